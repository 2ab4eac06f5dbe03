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
// so that only those under 2^-26 of the largest lose bits (a step is 2^-36 of
// it there).
//
// The kernel here is for few rows (up to 32 a sequence and kv head; the tiled
// one takes more): a wave decodes 64 keys and values straight into its operand
// registers, so every cached byte is read once and nothing goes through LDS
// but the queries.  A wave loads its next keys as soon as the first product
// has read the registers and its next values after the second; at D = 128
// three waves a SIMD (150 registers) hide the rest.  Memory bounds it: 64
// sequences of 2048 to 8192 tokens (8 kv heads, NVFP4 4/6, 379 MB) in 93 us
// of calls, 4.1 TB/s, where a large copy moves 4.85; 2 sequences up to 131072
// (MXFP4, 219 MB) in 53 us.  Vector instructions issue in 46% of the cycles.
// Short contexts are all latency: 2048 tokens of one sequence 7.3 us and 3.1
// to 4.1 for the join, in 10.4 us a call.
#pragma once

#include "kv_common.h"

namespace fp4q {

typedef __attribute__((address_space(4))) int32_t ConstInt;

struct AttnArgs {
  KvView c;
  const uint16_t* q;
  // constant address space: loads at wave-uniform places are scalar loads
  // whatever the kernel has stored, and do not wait for the vector loads
  const ConstInt *pt, *lens, *cu;
  uint16_t* out;
  float* lse;                            // [tokens][hq] or NULL
  float *po, *pm;                        // partials [splits][tokens][hq][D], [..][2] (max, sum)
  int* parts;                            // [tokens][hq] parts in use
  int64_t qs, os;                        // elements between tokens
  int64_t tokens, seqs, width;
  int hq, group, window, splits;
  uint32_t want;                         // workgroups wanted per kv head
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
// The bits of four scale bytes that count: an E4M3 scale's sign is ignored, by
// every decode of the library.
template <int MODE>
constexpr uint32_t kScaleBits = MODE == 2 ? 0xFFFFFFFFu : 0x7F7F7F7Fu;
// E4M3 scale bytes 2 HI and 2 HI + 1 of w as fp16 (exact).
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

// A workgroup's work: rows row0 .. row0 + M - 1 of sequence b, row r being
// token r / group with head r % group of the kv head's own, and part `split`
// of the `parts` that their context is cut into.  All rows together stay
// below 2^31.
struct Work {
  uint32_t b, tok0;                      // the sequence's first token
  uint32_t row0, rows;                   // rows of the whole sequence
  int len, n;                            // cached tokens, new ones
  uint32_t split, parts;
};

__device__ __forceinline__ uint32_t cu_at(const AttnArgs& a, uint32_t b) {
  const int v = a.cu[b];
  return v < 0 ? 0 : (v > (int)a.tokens ? (uint32_t)a.tokens : (uint32_t)v);
}

// Without parts, tile `t` of the grid: sequence b's tiles start at
// floor(cu[b] group / M) + b, which leaves room for every sequence's
// ceil(n group / M) whatever the n, so the grid needs no sizes from the
// device; ids between have no rows.  The search takes 64 boundaries at a
// time, one a lane.  Returns the tile of the sequence.
template <uint32_t M>
__device__ __forceinline__ uint32_t tile_of(const AttnArgs& a, uint32_t t, Work& w) {
  const uint32_t group = (uint32_t)a.group;
  if (!a.cu) {
    const uint32_t per = (group + M - 1) / M;
    w.b = t / per;
    return t - w.b * per;
  }
  uint32_t lo = 0, n = (uint32_t)a.seqs;             // the answer is in [lo, lo + n)
  while (n > 1) {
    const uint32_t step = (n + 63) / 64;
    const uint32_t at = step * (threadIdx.x & 63);
    const bool below = at < n && cu_at(a, lo + at) * group / M + lo + at <= t;
    const int k = __popcll(__ballot(below)) - 1;     // monotone: a prefix of the lanes
    const uint32_t skip = step * (uint32_t)(k < 0 ? 0 : k);
    lo += skip;
    n = n - skip < step ? n - skip : step;
  }
  w.b = __builtin_amdgcn_readfirstlane(lo);
  return t - (cu_at(a, w.b) * group / M + w.b);      // wraps to no tile before the first
}

// Blocks of 64 keys that a tile of `n` new tokens among `len` can reach.
__device__ __forceinline__ uint32_t blocks_in_reach(const AttnArgs& a, int64_t len, int64_t n) {
  const int64_t most = a.width << a.c.page_shift;
  int64_t reach = len > most ? most : len;
  if (a.window > 0 && reach > a.window + n) reach = a.window + n;
  return reach > 0 ? (uint32_t)((reach + kAttnKeys - 1) / kAttnKeys) : 0;
}

// Running sum over the wave by DPP: within rows of 16, then across.
template <int CTRL, int ROWS, typename T>
__device__ __forceinline__ T dpp_add(T v) {
  return v + __builtin_bit_cast(T, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL,
                                                               ROWS, 0xF, false));
}
template <typename T>
__device__ __forceinline__ T wave_prefix(T v) {      // inclusive
  v = dpp_add<0x111, 0xF>(v);            // row_shr 1, 2, 4, 8
  v = dpp_add<0x112, 0xF>(v);
  v = dpp_add<0x114, 0xF>(v);
  v = dpp_add<0x118, 0xF>(v);
  v = dpp_add<0x142, 0xA>(v);            // row_bcast 15 into rows 1 and 3
  return dpp_add<0x143, 0xC>(v);         // row_bcast 31 into rows 2 and 3
}
__device__ __forceinline__ uint32_t lane_value(uint32_t v, int lane) {
  return (uint32_t)__builtin_amdgcn_readlane((int)v, lane);
}

// With parts, item `t` of the list of (sequence, tile, part) in that order.  A
// sequence's context is cut into its share of a.want by blocks among the
// tiles of all sequences, so that every workgroup gets about the same number
// whatever the mixture of lengths (only the device knows them), but into at
// most a.splits parts of at least 4 blocks.  The list has no holes: hardware
// deals workgroups out to its engines in turn, and ids that ended at once at a
// fixed stride left whole engines idle (a prompt's 700 us became 2.8 ms).
template <uint32_t M>
__device__ __forceinline__ uint32_t item_of(const AttnArgs& a, uint32_t t, Work& w) {
  const uint32_t lane = threadIdx.x & 63, seqs = (uint32_t)a.seqs;
  uint32_t c0 = 0, n = 0, tiles = 0, blocks = 0;
  int len = 0;
  auto size = [&](uint32_t first) {      // sequence first + lane
    const uint32_t b = first + lane;
    const bool in = b < seqs;
    const uint32_t bb = in ? b : 0;
    len = a.lens[bb];
    c0 = b;
    n = in ? 1 : 0;
    if (a.cu) {
      c0 = cu_at(a, bb);
      const uint32_t c1 = cu_at(a, bb + 1);
      n = in && c1 > c0 ? c1 - c0 : 0;
    }
    tiles = (n * (uint32_t)a.group + M - 1) / M;
    blocks = blocks_in_reach(a, len, min(n, M / (uint32_t)a.group + 2));
  };
  float total = 0.0f;                    // tiles x blocks
  for (uint32_t first = 0; first < seqs; first += 64) {
    size(first);
    total += __uint_as_float(lane_value(__float_as_uint(wave_prefix((float)tiles * (float)blocks)), 63));
  }
  const float each = total > 0.0f ? (float)a.want / total : 0.0f;
  uint32_t before = 0;                   // items of the sequences before `first`
  for (uint32_t first = 0; first < seqs; first += 64) {
    if (seqs > 64) size(first);
    const uint32_t most = min((blocks + 3) / 4, (uint32_t)a.splits);
    const uint32_t parts = max(1u, min(most, (uint32_t)__builtin_rintf((float)blocks * each)));
    const uint32_t items = tiles * parts, upto = wave_prefix(items);
    const uint64_t past = __ballot(before + upto > t);
    if (past) {
      const int k = __builtin_ctzll(past);
      w.b = first + k;
      w.parts = lane_value(parts, k);
      w.tok0 = lane_value(c0, k);
      w.n = (int)lane_value(n, k);
      w.len = (int)lane_value((uint32_t)len, k);
      const uint32_t at = t - before - (lane_value(upto, k) - lane_value(items, k));
      const uint32_t tile = at / w.parts;
      w.split = at - tile * w.parts;
      return tile;
    }
    before += lane_value(upto, 63);
  }
  return ~0u;
}

// Rows r0 .. r1 - 1 of head h, counted from token tok0 on, that see nothing.
template <int D>
__device__ __forceinline__ void clear_rows(const AttnArgs& a, int h, uint32_t tok0, uint32_t r0,
                                           uint32_t r1) {
  uint32_t group = (uint32_t)a.group;
  asm volatile("" : "+s"(group));        // or its reciprocal stays in registers for good
  for (uint32_t i = threadIdx.x; i < (r1 - r0) * (D / 8); i += blockDim.x) {
    const uint32_t r = r0 + i / (D / 8), ch = i % (D / 8) * 8, tok = r / group;
    const int64_t t = tok0 + tok;
    const int head = (int)(h * group + (r - tok * group));
    *(uint4*)(a.out + t * a.os + (int64_t)head * D + ch) = make_uint4(0, 0, 0, 0);
    if (ch == 0 && a.lse) a.lse[t * a.hq + head] = -__builtin_inff();
  }
}

// Tokens before the first sequence and past the last one see nothing.  The
// tiles of the grid reach over them (tile_of: the first sequence's count back
// to token 0, the last one's up to the last token), so each clears the rows
// that no sequence has.  With parts the join does it.
template <int D, uint32_t M>
__device__ __forceinline__ void clear_gaps(const AttnArgs& a, int h, const Work& w, uint32_t next,
                                           uint32_t t, uint32_t tile) {
  const uint32_t group = (uint32_t)a.group;
  if (w.b == 0 && w.tok0 > 0) {
    const uint32_t end = w.tok0 * group;
    if ((uint64_t)t * M < end) clear_rows<D>(a, h, 0, t * M, min(end, t * M + M));
  }
  if (w.b + 1 == (uint32_t)a.seqs && next < (uint32_t)a.tokens && next >= w.tok0) {
    const uint32_t held = (next - w.tok0) * group, end = ((uint32_t)a.tokens - w.tok0) * group;
    if ((uint64_t)tile * M < end) {
      const uint32_t lo = max(held, tile * M), hi = min(end, tile * M + M);
      if (lo < hi) clear_rows<D>(a, h, w.tok0, lo, hi);
    }
  }
}

// The work of place `t` for one head; false where there is none.
template <int D, uint32_t M>
__device__ __forceinline__ bool find_work(const AttnArgs& a, int h, uint32_t t, Work& w) {
  uint32_t tile;
  if (a.splits > 1) {
    tile = item_of<M>(a, t, w);
    if (tile == ~0u) return false;
  } else {
    w.split = 0;
    w.parts = 1;
    tile = tile_of<M>(a, t, w);
    if (w.b >= (uint32_t)a.seqs) return false;
    w.tok0 = w.b;
    w.n = 1;
    if (a.cu) {
      w.tok0 = cu_at(a, w.b);
      const uint32_t next = cu_at(a, w.b + 1);
      w.n = next > w.tok0 ? (int)(next - w.tok0) : 0;
      clear_gaps<D, M>(a, h, w, next, t, tile);
    }
    w.len = a.lens[w.b];
  }
  w.rows = (uint32_t)w.n * (uint32_t)a.group;
  if ((uint64_t)tile * M >= w.rows) return false;
  w.row0 = tile * M;
  const int64_t most = a.width << a.c.page_shift;    // below 2^31
  if (w.len > most) w.len = (int)most;
  return true;
}

// Partial sums: [split][token][head], and how many parts a row has.
__device__ __forceinline__ int64_t row_at(const AttnArgs& a, const Work& w, int h, uint32_t row) {
  const uint32_t tok = row / (uint32_t)a.group;
  return (int64_t)(w.tok0 + tok) * a.hq + h * a.group + (row - tok * (uint32_t)a.group);
}
// Notes the parts of `count` rows; a part without blocks is an empty sum.
__device__ __forceinline__ void note_parts(const AttnArgs& a, const Work& w, int h, uint32_t count,
                                           bool empty, uint32_t threads) {
  for (uint32_t r = threadIdx.x; r < count && w.row0 + r < w.rows; r += threads) {
    const int64_t at = row_at(a, w, h, w.row0 + r);
    if (w.split == 0) a.parts[at] = (int)w.parts;
    if (empty) *(float2*)(a.pm + (w.split * a.tokens * a.hq + at) * 2) =
        make_float2(-__builtin_inff(), 0.0f);
  }
}

// One wave's share of 64 cached tokens: lane (c = lane & 15, g = lane >> 4)
// holds of keys 16 (c / 4) + 4 t + c % 4, t = 0..3, the channels D/4 g ..
// D/4 g + D/4 - 1, and of values the tokens 16 g .. 16 g + 15 of channel
// pairs 16 T + c.  The row order of the keys is what makes a lane's weights
// of the first product those of 16 consecutive tokens.
template <int MODE, int D>
struct KeyFragment {
  static constexpr int G = MODE == 2 ? 32 : 16;
  uint32_t k[4][D / 32], s[4];
};
template <int MODE, int D>
struct ValueFragment {
  u32x4_t v[D / 32], s[D / 32];
};

// Page ids of a lane's keys and values, -1 outside the cache or the table.
struct KvPages {
  int k, v;
};

// A sequence's row of the page table.  Keys, table width and pages stay below
// 2^31 (the host checks them), so a key's place is 32-bit arithmetic; keys of
// blocks past the end pass 2^31 by a few blocks at most and fit as unsigned.
struct PageRow {
  const ConstInt* row;
  uint32_t width, pages;
  int shift;
  __device__ __forceinline__ PageRow(const AttnArgs& a, uint32_t b)
      : row(a.pt + b * a.width), width((uint32_t)a.width), pages((uint32_t)a.c.pages),
        shift(a.c.page_shift) {}
  __device__ __forceinline__ int at(uint32_t key) const {
    const uint32_t i = key >> shift;
    if (i >= width) return -1;
    const uint32_t p = (uint32_t)row[i];
    return p < pages ? (int)p : -1;
  }
};

// With pages of 64 tokens and more a block lies in one page, whose address is
// the same for the whole wave (scalar arithmetic); with smaller ones each
// lane follows its own.
template <bool WIDE>
__device__ __forceinline__ KvPages load_pages(const PageRow& r, uint32_t base) {
  const int lane = (int)threadIdx.x & 63;
  KvPages p;
  if constexpr (WIDE) {
    p.k = p.v = r.at(base);
  } else {
    p.k = r.at(base + 16 * ((lane & 15) >> 2));
    p.v = r.at(base + 16 * (lane >> 4));
  }
  return p;
}

// Tokens before page `page` of head h, counted over the whole cache.
__device__ __forceinline__ int64_t head_page(const AttnArgs& a, int h, int page) {
  return (int64_t)((uint64_t)(uint32_t)(page < 0 ? 0 : page) * (uint32_t)a.c.heads + (uint32_t)h)
         << a.c.page_shift;
}

// N bytes at `base` + `lane` + `step`, the first (and the step) the same for
// the whole wave if WIDE: then through a buffer resource, whose base and
// offset are scalars, so that a block's addresses cost no vector arithmetic.
template <int N, bool WIDE>
struct KvLoad {
  typedef uint32_t T __attribute__((ext_vector_type(N >= 4 ? N / 4 : 1)));
  static __device__ __forceinline__ T at(const uint8_t* base, uint32_t lane, uint32_t step) {
    T v;
    if constexpr (WIDE) {
      // a page's part of one head is under 2^31 bytes (page_size * head_dim / 2 <= 2^19)
      const auto r = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(base), 0, 0x7FFFFFF0,
                                                       0x00020000);
      if constexpr (N == 16) v = __builtin_amdgcn_raw_buffer_load_b128(r, lane, step, 0);
      else if constexpr (N == 8) v = __builtin_amdgcn_raw_buffer_load_b64(r, lane, step, 0);
      else if constexpr (N == 4) v[0] = __builtin_amdgcn_raw_buffer_load_b32(r, lane, step, 0);
      else if constexpr (N == 2) v[0] = (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(r, lane, step, 0);
      else v[0] = (uint8_t)__builtin_amdgcn_raw_buffer_load_b8(r, lane, step, 0);
    } else {
      const uint8_t* p = base + lane + step;
      if constexpr (N >= 4) v = *(const T*)p;
      else if constexpr (N == 2) v[0] = *(const uint16_t*)p;
      else v[0] = *p;
    }
    return v;
  }
};

template <int MODE, int D, bool WIDE>
__device__ __forceinline__ void load_keys(const AttnArgs& a, int h, uint32_t base, KvPages pg,
                                          KeyFragment<MODE, D>& f) {
  constexpr int G = KeyFragment<MODE, D>::G, KD = D / 32;
  const int lane = (int)threadIdx.x & 63, c = lane & 15, g = lane >> 4;
  const uint32_t P = 1u << a.c.page_shift, seg = 16 * (c >> 2);
  // token of the page (the same for the wave when WIDE), and the lane's offset from it
  const int64_t at = head_page(a, h, pg.k) + ((WIDE ? base : base + seg) & (P - 1));
  const uint32_t row = (WIDE ? seg : 0) + (c & 3);
  const uint8_t* kc = a.c.kc + at * (D / 2);
  const uint8_t* ks = a.c.ks + at * (D / G);
  const uint32_t ko = row * (D / 2) + g * (D / 8), so = row * (D / G) + g * (D / 4) / G;
  constexpr int KB = KD * 4 > 16 ? 16 : KD * 4;      // bytes of a load
  constexpr int SB = D / 4 >= G ? D / 4 / G : 1;     // scale bytes of a lane's channels
#pragma unroll
  for (int t = 0; t < 4; t++) {
#pragma unroll
    for (int i = 0; i < KD; i += KB / 4) {
      const auto w = KvLoad<KB, WIDE>::at(kc, ko + (t * 4 * (D / 2) + i * 4), 0);
#pragma unroll
      for (int e = 0; e < KB / 4; e++) f.k[t][i + e] = w[e];
    }
    f.s[t] = KvLoad<SB, WIDE>::at(ks, so + t * 4 * (D / G), 0)[0];
  }
}

template <int MODE, int D, bool WIDE>
__device__ __forceinline__ void load_values(const AttnArgs& a, int h, uint32_t base, KvPages pg,
                                            ValueFragment<MODE, D>& f) {
  constexpr int G = KeyFragment<MODE, D>::G, KD = D / 32;
  const int lane = (int)threadIdx.x & 63, c = lane & 15, g = lane >> 4;
  const uint32_t P = 1u << a.c.page_shift;
  const int64_t pv = head_page(a, h, pg.v);
  const uint32_t at = (WIDE ? base : base + 16 * g) & (P - 1), tok = WIDE ? 16 * g : 0;
  const uint8_t* vc = a.c.vc + pv * (D / 2) + at;
  const uint8_t* vs = a.c.vs + pv * (D / G) + at;
  const uint32_t vo = ((uint32_t)c << a.c.page_shift) + tok;
  const uint32_t so = ((uint32_t)(MODE == 2 ? 0 : c >> 3) << a.c.page_shift) + tok;
#pragma unroll
  for (int T = 0; T < KD; T++) {
    f.v[T] = KvLoad<16, WIDE>::at(vc, vo, (uint32_t)(16 * T) << a.c.page_shift);
    f.s[T] = KvLoad<16, WIDE>::at(vs, so, (uint32_t)(MODE == 2 ? T : 2 * T) << a.c.page_shift);
  }
}

// A operand of key rows: 8 channels of code dword `w` and the lane's scales (of
// kScaleBits).
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
// tokens of dwords w0, w1 with their scale bytes s0, s1 (of kScaleBits).
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

// Queries of one column as B operands of NS steps, each lane's 8 channels of
// step s at q + s * STRIDE; `reduce` takes a maximum over the column's lanes.
// Returns the factor that turns the products into scores in powers of two.
// A scale of 0 makes every score 0; a negative one goes to the queries, so
// that the factor is positive.
template <int MODE, int NS, int STRIDE, typename R>
__device__ __forceinline__ float load_query(const AttnArgs& a, int h, const uint16_t* q,
                                            u32x4_t (&o)[NS], R&& reduce) {
  const float k = fabsf(a.scale) * kLog2e;
  const uint32_t keep = a.scale == 0.0f ? 0u : ~0u, flip = a.scale < 0.0f ? 0x80008000u : 0u;
#pragma unroll
  for (int s = 0; s < NS; s++) o[s] = *(const u32x4_t*)(q + s * STRIDE);
  if (keep == 0 || flip) {
#pragma unroll
    for (int s = 0; s < NS; s++) o[s] = (o[s] & keep) ^ flip;
  }
  if constexpr (MODE == 2) {
    return fmaxf(k, 0x1p-126f);
  } else {
    uint32_t m = 0;
#pragma unroll
    for (int s = 0; s < NS; s++)
#pragma unroll
      for (int i = 0; i < 4; i++)
        m = max(m, max(o[s][i] & 0x7FFFu, (o[s][i] >> 16) & 0x7FFFu));
    const float top = reduce(__uint_as_float(m << 16));
    int shift = 141 - (int)(__float_as_uint(top) >> 23);         // 2^14 <= top 2^shift < 2^15
    shift = shift > 127 ? 127 : shift;
#pragma unroll
    for (int s = 0; s < NS; s++)
#pragma unroll
      for (int i = 0; i < 4; i++)
        o[s][i] = bits_of(f16x2_t{(_Float16)__builtin_ldexpf(bf16_lo(o[s][i]), shift),
                                  (_Float16)__builtin_ldexpf(bf16_hi(o[s][i]), shift)});
    const float alpha = a.c.kam[h] / (6.0f * (MODE == 1 ? 256.0f : 448.0f));
    return fmaxf(__builtin_ldexpf(k * alpha, -shift), 0x1p-126f);
  }
}

// Scores from the products x: in powers of two, s = f x + off with f > 0, so
// that maxima can be taken of x and the weight is one fma and one exponential.
//
// Capped ones, c tanh(t) with t = s / c, have two forms:
//  - caps up to kShortCap: c - 2 c / (exp(2 t) + 1), so x = -1 / (exp + 1)
//    takes the place of the product, f = 2 c and off = c.  Its roundings are
//    relative to c: 8 u c at most (u = 2^-24), 3e-5 of a weight at 64.
//  - larger ones, whose scores lie around zero more often than not: x stays
//    the product times tanh(t) / t, so the error follows the score.  Up to
//    |t| = 0.3 that ratio is its series to t^8 (the first term left out is
//    under u), beyond x = `top` (1 - 2 / (exp(2 t) + 1)), 16 u of the score.
// Every score of the short form costs two transcendentals and two other
// instructions, of the other one about nine more: a prompt of 8192 tokens with
// a window of 4096 takes 481 us under a cap of 64 and 686 under one of 100,
// chunks of 512 tokens over 6144 163 and 281, 64 decoding contexts 92 and 98.
constexpr float kShortCap = 64.0f;
struct ScoreScale {
  float f, off, in;                      // in > 0: capped; 2 t in powers of two = in x
};
__device__ __forceinline__ ScoreScale score_scale(const AttnArgs& a, float qf) {
  constexpr float kMax = 3.402823466e38f;
  ScoreScale s{qf, 0.0f, 0.0f};
  if (a.cap > 0.0f) {
    // finite for the least of caps, so that a product of 0 stays 0
    s.in = fminf(qf * fminf(2.0f / a.cap, kMax), kMax);
    if (a.cap <= kShortCap) {
      s.f = fmaxf(2.0f * a.cap * kLog2e, 0x1p-126f);
      s.off = a.cap * kLog2e;
    }
  }
  return s;
}
__device__ __forceinline__ float capped_short(float x, float in) {
  return __builtin_amdgcn_rcpf(-1.0f - __builtin_amdgcn_exp2f(x * in));
}
__device__ __forceinline__ float capped_long(float x, float in, float top) {
  constexpr float k = 1.0f / (4.0f * kLog2e * kLog2e);           // t^2 = k y^2
  const float y = x * in, z = y * y * k;
  float r = __builtin_fmaf(z, 62.0f / 2835.0f, -17.0f / 315.0f);
  r = __builtin_fmaf(z, r, 2.0f / 15.0f);
  r = __builtin_fmaf(z, r, -1.0f / 3.0f);
  r = __builtin_fmaf(z * r, x, x);
  const float far = top * __builtin_fmaf(
      -2.0f, __builtin_amdgcn_rcpf(__builtin_amdgcn_exp2f(y) + 1.0f), 1.0f);
  return z < 0.09f ? r : far;
}
// A lane's capped scores (a vector of floats).
template <bool LONG, typename V>
__device__ __forceinline__ void cap_scores(const ScoreScale& sc, V& s) {
  constexpr int N = sizeof(V) / sizeof(float);
  if constexpr (LONG) {
    const float top = fminf(2.0f * kLog2e / sc.in, 3.402823466e38f);       // c / f
#pragma unroll
    for (int r = 0; r < N; r++) s[r] = capped_long(s[r], sc.in, top);
  } else {
#pragma unroll
    for (int r = 0; r < N; r++) s[r] = capped_short(s[r], sc.in);
  }
}

// The weight of a score is exp2(f x - (m - off - kOff)) in one fma, whose exact
// product keeps what m lost in its rounding: a sixteenth at kFarMax, but from
// about 2^25 on more than the weights' exponents hold.  Past kFarMax a lane's
// scores are rounded as m was and replaced by their distances to it, over f, so
// that the same fma with the reference -kOff gives the weight.
constexpr float kFarMax = 0x1p20f;
template <typename V>
__device__ __forceinline__ void far_scores(const ScoreScale& sc, float m, V& s) {
  const float rf = __builtin_amdgcn_rcpf(sc.f);
#pragma unroll
  for (int r = 0; r < (int)(sizeof(V) / sizeof(float)); r++)
    s[r] = (__builtin_fmaf(s[r], sc.f, sc.off) - m) * rf;
}

// NT columns of 16 query rows, WAVES waves that take the blocks of 64 keys of
// the workgroup's part of the context in turn and join their sums at the end.
template <int MODE, int D, int NT, int WAVES, bool WIDE>
__global__ __launch_bounds__(64 * WAVES, D == 256 || NT == 2 ? 2 : (D == 128 ? 3 : 4))
void kv_attention_kernel(AttnArgs a) {
  constexpr int KD = D / 32, M = 16 * NT;
  constexpr float kOff = MODE == 2 ? 0.0f : 12.0f;   // weights carry 2^kOff
  // the running maximum may lag by 2^kLag before everything is rescaled (fp16
  // weights then stay under 2^15; bf16 and the sums have room)
  constexpr float kLag = MODE == 2 ? 8.0f : 3.0f;
  __shared__ float so[WAVES][16][D + 4];
  __shared__ float sm[WAVES][16][2];
  __shared__ u32x4_t sq[NT][KD][64];     // the queries, each lane's operand (registers are short)
  const int lane = (int)threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int c = lane & 15, g = lane >> 4;
  // heads fastest: consecutive ids go to consecutive XCDs
  const uint32_t place = blockIdx.x / (uint32_t)a.c.heads;
  const int h = (int)(blockIdx.x - place * (uint32_t)a.c.heads);
  Work rt;
  if (!find_work<D, M>(a, h, place, rt)) return;
  const int split = (int)rt.split;
  // reach of the tile's rows: [lo, hi) of each column, and of all together
  const uint32_t group = (uint32_t)a.group;
  const uint32_t last = rt.rows - rt.row0 > M ? rt.row0 + M - 1 : rt.rows - 1;
  auto hi_of = [&](uint32_t row) {
    const int64_t x = (int64_t)rt.len - rt.n + row / group + 1;
    return (int)(x < 0 ? 0 : x);
  };
  auto lo_of = [&](int hi) { return a.window > 0 && hi > a.window ? hi - a.window : 0; };
  const int hmin = hi_of(rt.row0), hmax = hi_of(last);
  const int lmin = lo_of(hmin), lmax = lo_of(hmax);
  const uint32_t base0 = (uint32_t)lmin & ~(uint32_t)(kAttnKeys - 1);
  const uint32_t blocks = a.c.pages > 0 && hmax > lmin ? ((uint32_t)hmax - base0 + kAttnKeys - 1) / kAttnKeys : 0;
  const uint32_t per = (blocks + rt.parts - 1) / rt.parts;
  const uint32_t end = (split + 1) * per < blocks ? (split + 1) * per : blocks;
  if (a.splits > 1) {
    const bool empty = split * per >= blocks;
    note_parts(a, rt, h, M, empty, 64 * WAVES);
    if (empty) return;
  }
  int hi[NT], lo[NT];
  ScoreScale sc[NT];
  float m[NT], l[NT];
  f32x4_t o[NT][KD][2];
#pragma unroll
  for (int i = 0; i < NT; i++) {
    // columns past the last row repeat it; their results are not stored
    const uint32_t row = min(rt.row0 + 16 * i + c, rt.rows - 1), tok = row / group;
    hi[i] = hi_of(row);
    lo[i] = lo_of(hi[i]);
    const uint16_t* x = a.q + (int64_t)(rt.tok0 + tok) * a.qs +
                        (int64_t)(h * group + row - tok * group) * D + g * (D / 4);
    u32x4_t q[KD];
    sc[i] = score_scale(a, load_query<MODE, KD, 8>(a, h, x, q, col_max));
    if (wave == 0) {
#pragma unroll
      for (int st = 0; st < KD; st++) sq[i][st][lane] = q[st];
    }
    m[i] = -__builtin_inff();
    l[i] = 0.0f;
#pragma unroll
    for (int T = 0; T < KD; T++) o[i][T][0] = o[i][T][1] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
  }
  uint32_t blk = split * per + wave;

  KeyFragment<MODE, D> kf;
  ValueFragment<MODE, D> vf;
  const PageRow pages(a, rt.b);
  auto base_of = [&](uint32_t i) { return base0 + i * kAttnKeys; };
  // one block: its keys and values are in kf and vf; the next block's loads go out
  // as soon as the registers are free, keys after the first product, values
  // after the second
  auto step = [&](uint32_t base, KvPages pg, bool more, uint32_t next, KvPages npg) {
    f32x4_t s[NT][4];
#pragma unroll
    for (int i = 0; i < NT; i++)
#pragma unroll
      for (int t = 0; t < 4; t++) s[i][t] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
    u32x4_t q[NT][KD];
    int opaque;                          // so that these reads stay in the loop
    asm volatile("v_mov_b32 %0, %1" : "=v"(opaque) : "v"(lane));
#pragma unroll
    for (int i = 0; i < NT; i++)
#pragma unroll
      for (int st = 0; st < KD; st++) q[i][st] = sq[i][st][opaque];
    static_for<4>([&](auto tt) {
      constexpr int t = decltype(tt)::value;
      static_for<KD>([&](auto ss) {
        constexpr int st = decltype(ss)::value;
        const u32x4_t k = key_operand<MODE, st * 8 / KeyFragment<MODE, D>::G>(
            kf.k[t][st], kf.s[t] & kScaleBits<MODE>);
#pragma unroll
        for (int i = 0; i < NT; i++) s[i][t] = mfma16<MODE>(k, q[i][st], s[i][t]);
      });
    });
    if (more) load_keys<MODE, D, WIDE>(a, h, next, npg, kf);
    if (a.cap > 0.0f) {
#pragma unroll
      for (int i = 0; i < NT; i++)
#pragma unroll
        for (int t = 0; t < 4; t++) {
          if (a.cap > kShortCap) cap_scores<true>(sc[i], s[i][t]);
          else cap_scores<false>(sc[i], s[i][t]);
        }
    }
    constexpr uint32_t kAll = kScaleBits<MODE>;
    uint32_t keep[4] = {kAll, kAll, kAll, kAll};     // scale bits of the tokens that count
    if (base < (uint32_t)lmax || base + kAttnKeys > (uint32_t)hmin || !__all(pg.v >= 0)) {
#pragma unroll
      for (int t = 0; t < 4; t++) {
        keep[t] = 0;
#pragma unroll
        for (int r = 0; r < 4; r++) {
          const int key = (int)base + 16 * g + 4 * t + r;
          if (pg.v >= 0 && key >= lmin && key < hmax) keep[t] |= kAll & 255u << (8 * r);
#pragma unroll
          for (int i = 0; i < NT; i++)
            s[i][t][r] = pg.v < 0 || key < lo[i] || key >= hi[i] ? -__builtin_inff() : s[i][t][r];
        }
      }
    }
    u32x4_t p[NT][2];
#pragma unroll
    for (int i = 0; i < NT; i++) {
      float mx = s[i][0][0];
#pragma unroll
      for (int t = 0; t < 4; t++)
#pragma unroll
        for (int r = 0; r < 4; r++) mx = fmaxf(mx, s[i][t][r]);
      mx = fmaxf(m[i], __builtin_fmaf(col_max(mx), sc[i].f, sc[i].off));
      if (__any(mx > m[i] + kLag)) {
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
      float ref = (m[i] == -__builtin_inff() ? 0.0f : m[i]) - kOff - sc[i].off;
      if (fabsf(ref) > kFarMax) {
#pragma unroll
        for (int t = 0; t < 4; t++) far_scores(sc[i], m[i], s[i][t]);
        ref = -kOff;
      }
#pragma unroll
      for (int t = 0; t < 4; t++) {
        float e[4];
#pragma unroll
        for (int r = 0; r < 4; r++) {
          e[r] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[i][t][r], sc[i].f, -ref));
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
        value_operands<MODE>(vf.v[T][2 * u], vf.v[T][2 * u + 1], vf.s[T][2 * u] & keep[2 * u],
                             vf.s[T][2 * u + 1] & keep[2 * u + 1], even, odd);
#pragma unroll
        for (int i = 0; i < NT; i++) {
          o[i][T][0] = mfma16<MODE>(even, p[i][u], o[i][T][0]);
          o[i][T][1] = mfma16<MODE>(odd, p[i][u], o[i][T][1]);
        }
      }
    if (more) load_values<MODE, D, WIDE>(a, h, next, npg, vf);
  };

  __syncthreads();                       // the queries are in LDS
  if (blk < end) {
    KvPages pg = load_pages<WIDE>(pages, base_of(blk));
    KvPages npg = load_pages<WIDE>(pages, base_of(blk + WAVES));
    load_keys<MODE, D, WIDE>(a, h, base_of(blk), pg, kf);
    __builtin_amdgcn_sched_barrier(0);   // keys first, as in the loop: its waits count on it
    load_values<MODE, D, WIDE>(a, h, base_of(blk), pg, vf);
    for (; blk < end; blk += WAVES) {
      const KvPages after = load_pages<WIDE>(pages, base_of(blk + 2 * WAVES));
      step(base_of(blk), pg, blk + WAVES < end, base_of(blk + WAVES), npg);
      pg = npg;
      npg = after;
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
      const uint32_t full = rt.row0 + 16 * i + rr;
      if (full >= rt.rows) break;
      float mw[WAVES], ll = 0.0f, top = -__builtin_inff();
#pragma unroll
      for (int w = 0; w < WAVES; w++) top = fmaxf(top, mw[w] = sm[w][rr][0]);
#pragma unroll
      for (int w = 0; w < WAVES; w++)
        ll += sm[w][rr][1] * (mw[w] == top ? 1.0f : __builtin_amdgcn_exp2f(mw[w] - top));
      const int64_t tk = rt.tok0 + full / group;
      const int hd = (int)(h * group + full % group);
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

// Joins the parts of the context: D/4 lanes (16 bytes each) times
// `groups` (a power of two) for a query row, the groups taking its parts in
// turn.
template <int MODE, int D>
__global__ __launch_bounds__(kThreads) void kv_attention_join_kernel(AttnArgs a, int groups, bool eager) {
  constexpr float kOff = MODE == 2 ? 0.0f : 12.0f;
  constexpr int L = D / 4;
  __shared__ float4 sx[kThreads];
  __shared__ float2 sm[kThreads];
  const int t = (int)threadIdx.x, lane = t % L, grp = t / L % groups;
  const int64_t row = (int64_t)blockIdx.x * (kThreads / (L * groups)) + t / (L * groups);
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
    // with few rows the loads do not wait for the number of parts (sums that
    // were not written are read and dropped): the call is all latency
    // Rows of no sequence have no number of parts: theirs is whatever the
    // workspace held.
    const uint32_t at = (uint32_t)row / (uint32_t)a.hq;
    const bool held = !a.cu || (at >= cu_at(a, 0) && at < cu_at(a, (uint32_t)a.seqs));
    const int n = held ? min(max(a.parts[row], 0), a.splits) : 0, most = eager ? a.splits : n;
    for (int s0 = grp; s0 < most; s0 += 4 * groups) {
      float2 ml[4];
      float4 y[4];
#pragma unroll
      for (int e = 0; e < 4; e++) {
        const int64_t s = s0 + e * groups;
        if (s >= most) continue;
        ml[e] = *(const float2*)(a.pm + (s * rows + row) * 2);
        y[e] = *(const float4*)(a.po + (s * rows + row) * D + lane * 4);
      }
      if (s0 >= n) break;
#pragma unroll
      for (int e = 0; e < 4; e++)
        if (s0 + e * groups < n && ml[e].y != 0.0f) add(ml[e].x, ml[e].y, y[e]);
    }
  }
  if (groups > 1) {
    for (int half = groups / 2; half > 0; half >>= 1) {
      __syncthreads();
      sx[t] = make_float4(x[0], x[1], x[2], x[3]);
      sm[t] = make_float2(top, l);
      __syncthreads();
      if (grp < half) add(sm[t + half * L].x, sm[t + half * L].y, sx[t + half * L]);
    }
  }
  if (!live || grp) return;
  const int64_t tok = (uint32_t)row / (uint32_t)a.hq;
  const int head = (int)(row - tok * a.hq), h = (int)((uint32_t)head / (uint32_t)a.group);
  const float va = MODE == 2 ? 1.0f : a.c.vam[h] / (6.0f * (MODE == 1 ? 256.0f : 448.0f));
  const float inv = l == 0.0f ? 0.0f : va / l;
  *(uint2*)(a.out + tok * a.os + (int64_t)head * D + lane * 4) =
      make_uint2(bf16x2_of(x[0] * inv, x[1] * inv), bf16x2_of(x[2] * inv, x[3] * inv));
  if (a.lse && lane == 0)
    a.lse[row] = l == 0.0f ? -__builtin_inff() : __builtin_fmaf(top - kOff, kLn2, logf(l));
}

}  // namespace fp4q
