// feedforward.h -- entry points of the feed-forward operators (products with
// FP4 weights, routing, experts, the norms around a block), compiled as part of
// fp4q.hip: argument checks on the host, then kernel launches on the caller's
// stream.  See include/fp4q.h for the contract.
#pragma once

#include <hip/hip_runtime.h>

#include <cmath>
#include <type_traits>

#include "experts_kernels.h"
#include "host_common.h"
#include "linear_kernels.h"
#include "linear_stream_kernels.h"
#include "linear_tiled_kernels.h"
#include "residual_kernels.h"
#include "route_kernels.h"

namespace fp4q {
namespace feedforward {

// ------------------------------------------------------------------ weights
inline int check_weights(const fp4_weights* w) {
  if (!w) return FP4_E_NULL;
  if (w->format != FP4_FORMAT_NVFP4 && w->format != FP4_FORMAT_MXFP4) return FP4_E_FLAGS;
  const bool nv = w->format == FP4_FORMAT_NVFP4;
  if (w->flags & ~(uint32_t)(nv ? FP4_BLOCK2D | FP4_ROW_ALPHA : 0)) return FP4_E_FLAGS;
  constexpr int64_t most = (int64_t)1 << 24;
  if (w->experts < 0 || w->experts > most || w->rows < 0 || w->rows >= most || w->cols < 0 ||
      w->cols >= most / 4 || w->cols % 32 || ((w->flags & FP4_BLOCK2D) && w->rows % 16))
    return FP4_E_SHAPE;
  if (w->rows > 0 && w->cols > 0 && w->experts > kMaxElems / (w->rows * w->cols)) return FP4_E_SHAPE;
  if (w->experts * w->rows == 0) return FP4_OK;
  if ((w->cols && (!w->codes || !w->scales)) || (nv && !w->alpha)) return FP4_E_NULL;
  return aligned(w->codes, 16) && aligned(w->scales, 2) && aligned(w->alpha, 4) ? FP4_OK : FP4_E_ALIGN;
}

inline WeightView weight_view(const fp4_weights* w) {
  const bool nv = w->format == FP4_FORMAT_NVFP4, tiles = w->flags & FP4_BLOCK2D;
  const bool by_row = w->flags & FP4_ROW_ALPHA;
  WeightView v;
  v.codes = w->codes;
  v.scales = w->scales;
  v.alpha = nv ? w->alpha : nullptr;
  v.codes_e = w->rows * (w->cols / 2);
  v.scales_e = (tiles ? w->rows / 16 : w->rows) * (w->cols / (nv ? 16 : 32));
  v.alpha_e = by_row ? w->rows : 1;
  v.rows = (int)w->rows;
  v.cols = (int)w->cols;
  v.tile_shift = tiles ? 4 : 0;
  v.row_alpha = by_row;
  return v;
}

// The kernels address rows of x in 31 bits: 128 of them stay within.
constexpr int64_t kMaxXStride = (int64_t)1 << 23;

// Rows of `width` elements, `stride` apart.
inline int check_rows(int64_t tokens, int64_t stride, int64_t width, int64_t multiple) {
  if (stride < width || stride % multiple || stride >= kMaxElems) return FP4_E_SHAPE;
  return tokens > 0 && stride > kMaxElems / tokens ? FP4_E_SHAPE : FP4_OK;
}

// f(first, count) for slices of the tokens, one after another, each of as many as a
// launch of workgroups of `threads` threads and `per_group` tokens can have.
template <typename F>
hipError_t in_slices(int64_t tokens, int64_t per_group, int64_t threads, F&& f) {
  const int64_t most = kMaxThreads / threads * per_group;
  hipError_t err = hipSuccess;
  for (int64_t t = 0; t < tokens && err == hipSuccess; t += most)
    err = f(t, tokens - t < most ? tokens - t : most);
  return err;
}

// Tokens of a slice of a product with `rows` rows: the forms' launches stay within
// kMaxThreads (32 threads a token and 128 rows at most, with as many left over).
inline int64_t linear_slice(int64_t rows) {
  const int64_t most = ((int64_t)1 << 33) / rows & ~(int64_t)127;
  return most < (1 << 24) ? most : 1 << 24;
}

// ------------------------------------------------------------------ few tokens
// Waves that share a row's K, the fewest that give every CU two workgroups (or
// have a step of K each): fewer meet in fewer joins.
inline void cut_rows(ColsArgs& a, int rows, int64_t slots, int r, int waves) {
  const int steps = (a.w.cols + kColsStep - 1) / kColsStep;
  a.wk = 1;
  while (a.wk < waves && a.wk < steps && cdiv(rows, 16 * r * (waves / a.wk)) * slots * waves < 16 * num_cus())
    a.wk *= 2;
  a.row_blocks = (int)cdiv(rows, 16 * r * (waves / a.wk));
}

template <int R, bool GATED, int SRC>
hipError_t launch_cols(int format, ColsArgs a, int64_t slots, hipStream_t st) {
  constexpr int W = SRC == kDense ? 8 : 4;
  cut_rows(a, GATED ? a.inner : a.w.rows, slots, R, W);
  const int64_t grid = slots * a.row_blocks;
  if (grid >= ((int64_t)1 << 31)) return hipErrorInvalidConfiguration;
  return format == FP4_FORMAT_NVFP4
             ? launch(fp4_cols_kernel<0, R, GATED, SRC, W>, (unsigned)grid, W * 64, st, a)
             : launch(fp4_cols_kernel<1, R, GATED, SRC, W>, (unsigned)grid, W * 64, st, a);
}

// Streams of codes read scales in whole dwords.
inline bool stream_fits(const fp4_weights* w) {
  return w->cols % (w->format == FP4_FORMAT_NVFP4 ? 64 : 128) == 0 && aligned(w->scales, 4);
}

// busy: workgroups' worth of experts that can have tokens; tokens: an upper bound
// of an expert's where no token names it twice, for which a segment is sized.
// Where rows are few their K is cut until every CU has a
// workgroup.  Where they are many a workgroup takes several blocks, up to four
// rounds of workgroups, since experts have unequal numbers of tokens (64 tokens
// through 128 experts, gate and up: 1 round 161 us, 2 131, 4 120, 8 120).
template <bool GATED, int SRC>
hipError_t launch_stream(int format, ColsArgs a, int64_t slots, int64_t busy, int64_t tokens,
                         hipStream_t st) {
  const int64_t rows = GATED ? a.inner : a.w.rows, wave_rows = GATED ? 16 : 32;
  const StreamSegment seg = stream_segment(tokens, a.w.cols);
  a.kseg_shift = seg.shift;
  a.span = seg.span;
  a.wk = 1;
  while (a.wk < kStreamWaves && 1024 * a.wk <= (1 << seg.shift) && 512 * a.wk < a.w.cols &&
         cdiv(rows, wave_rows * (kStreamWaves / a.wk)) * busy < num_cus())
    a.wk *= 2;
  const int64_t all = cdiv(rows, wave_rows * (kStreamWaves / a.wk));
  const int64_t each = a.wk == 1 ? all * busy / (8 * num_cus()) : 1;
  a.blocks = (int)(each < 1 ? 1 : (each < all ? each : all));
  a.row_blocks = (int)cdiv(all, a.blocks);
  const int64_t grid = slots * a.row_blocks;
  if (grid >= ((int64_t)1 << 31)) return hipErrorInvalidConfiguration;
  return format == FP4_FORMAT_NVFP4
             ? launch(fp4_stream_kernel<0, GATED, SRC>, (unsigned)grid, kStreamThreads, st, a)
             : launch(fp4_stream_kernel<1, GATED, SRC>, (unsigned)grid, kStreamThreads, st, a);
}

// 16 NT tokens at a time; waves share rows where a workgroup's 256 leave CUs idle.
template <int NT>
hipError_t launch_mid(int format, ColsArgs a, hipStream_t st) {
  const int64_t slots = cdiv(a.tokens, 16 * NT);
  a.wk = 1;
  while (a.wk < 4 && cdiv(a.w.rows, 32 * (kMidWaves / a.wk)) * slots < num_cus()) a.wk *= 2;
  a.row_blocks = (int)cdiv(a.w.rows, 32 * (kMidWaves / a.wk));
  const int64_t grid = slots * a.row_blocks;
  if (grid >= ((int64_t)1 << 31)) return hipErrorInvalidConfiguration;
  return format == FP4_FORMAT_NVFP4
             ? launch(fp4_mid_kernel<0, NT>, (unsigned)grid, kMidThreads, st, a)
             : launch(fp4_mid_kernel<1, NT>, (unsigned)grid, kMidThreads, st, a);
}

// ------------------------------------------------------------------ many tokens
template <bool GATED, bool EXPERTS>
hipError_t launch_tiled(int format, TiledArgs a, hipStream_t st) {
  a.tiles_n = (uint32_t)cdiv(GATED ? a.inner : a.w.rows, GATED ? kTileWeights / 2 : kTileWeights);
  const int64_t grid = EXPERTS ? cdiv(a.tiles_t, 4 * kXcds) * 4 * kXcds * a.tiles_n
                               : xcd_grid(a.tiles_t, a.tiles_n, 8, 8);
  if (grid >= ((int64_t)1 << 31)) return hipErrorInvalidConfiguration;
  return format == FP4_FORMAT_NVFP4
             ? launch(fp4_tiled_kernel<0, GATED, EXPERTS>, (unsigned)grid, kTiledThreads, st, a)
             : launch(fp4_tiled_kernel<1, GATED, EXPERTS>, (unsigned)grid, kTiledThreads, st, a);
}

// What the two forms of a call have in common.
inline TiledArgs tiled_args(const ColsArgs& a) {
  TiledArgs t = {};
  t.w = a.w;
  t.x = a.x;
  t.out = a.out;
  t.xs = a.xs;
  t.os = a.os;
  t.tokens = a.tokens;
  t.off = a.off;
  t.order = a.order;
  t.top_k = a.top_k;
  t.experts = a.experts;
  t.inner = a.inner;
  t.x_per_token = a.x_per_token;
  t.x_bytes = a.x_bytes;
  t.out_f32 = a.out_f32;
  return t;
}

// Tiles of 16 tokens that a workgroup takes: the fewest with which all workgroups
// of 64 rows run at once, for the shorter way of each; past that as many as fit.
inline int linear_tiles(int64_t tokens, int64_t rows) {
  for (int nt = 1; nt < 4; nt++)
    if (cdiv(tokens, 16 * nt) * cdiv(rows, 64) <= num_cus()) return nt;
  return 4;
}

// Streams for matrices of many rows, the more the more tokens: a workgroup waits for
// all of its activations first (4096 columns of NVFP4, streams and cols: 1 token of
// 4096 rows 8.6 and 7.6 us, 8192 8.7 and 9.2, 28672 19.4 and 24.5; 8 tokens 8192 12.6
// and 9.7, 14336 13.9 and 15.5; 16 tokens 14336 23.3 and 17.8, 28672 24.3 and 31.5).
inline bool streams_sooner(const fp4_weights* w, int64_t tokens) {
  return w->rows >= 8192 && w->rows >= 1792 * tokens && w->cols > 0 && stream_fits(w);
}

// Two row tiles a wave, so that a token's activations are read for 32 rows at a
// time, where that leaves work for three CUs of four (16 tokens through 14336x4096
// 17.8 us, one tile 24.4; through 4096x4096 10.8 and 8.6).
inline bool tall(int64_t rows, int64_t slots) {
  return cdiv(rows, 32) * slots * 4 >= 3 * (int64_t)num_cus();
}

// A round of 128x256 tiles, one a CU, takes as long as six and a half of 64 tokens
// x 64 rows (88 us and 14 with 4096 columns): whichever has done sooner.  Of several
// rounds two tiles share a CU and take less than twice as long (256 tiles 94 us, 512
// 139, 1024 290), far beyond the sizes at which the two forms meet.
inline bool tiles_sooner(int64_t tokens, int64_t rows) {
  const int64_t tiles = cdiv(tokens, kTileTokens) * cdiv(rows, kTileWeights);
  const int64_t mids = cdiv(tokens, 64) * cdiv(rows, 64);
  return tokens > 64 && 13 * cdiv(tiles, num_cus()) <= 2 * cdiv(mids, num_cus());
}

// A slice of a product's tokens.
inline hipError_t linear_call(const fp4_weights* w, const uint16_t* x, int64_t x_stride,
                              int64_t tokens, void* out, int64_t out_stride, bool out_f32,
                              hipStream_t st) {
  ColsArgs a = {};
  a.w = weight_view(w);
  a.x = x;
  a.out = out;
  a.xs = x_stride;
  a.os = out_stride;
  a.tokens = tokens;
  a.out_f32 = out_f32;
  a.out_vec = out_stride % 4 == 0 && aligned(out, out_f32 ? 16 : 8);
  if (w->cols > 0 && tiles_sooner(tokens, w->rows)) {
    TiledArgs t = tiled_args(a);
    t.tiles_t = (uint32_t)cdiv(tokens, kTileTokens);
    t.out_vec = out_stride % (out_f32 ? 4 : 8) == 0 && aligned(out, 16);
    return launch_tiled<false, false>(w->format, t, st);
  }
  if (tokens <= 16 && streams_sooner(w, tokens))
    return launch_stream<false, kDense>(w->format, a, 1, 1, tokens, st);
  if (tokens <= 16 || w->cols < kMidLeast) {
    const int64_t slots = cdiv(tokens, 16);
    return tall(w->rows, slots) ? launch_cols<2, false, kDense>(w->format, a, slots, st)
                                : launch_cols<1, false, kDense>(w->format, a, slots, st);
  }
  switch (linear_tiles(tokens, w->rows)) {
    case 1: return launch_mid<1>(w->format, a, st);
    case 2: return launch_mid<2>(w->format, a, st);
    case 3: return launch_mid<3>(w->format, a, st);
    default: return launch_mid<4>(w->format, a, st);
  }
}

// ------------------------------------------------------------------ experts
// The tiled kernel addresses its rows of x and h in 31 bits: batches past that
// go in slices of tokens, one after another in the same workspace.
constexpr int64_t kSliceBytes = 0x7FFF0000;

// More tokens an expert than streams, 16 at a time, are worth (64 and 128 experts,
// NVFP4: 16 tokens each 186 us by streams, 257 by tiles, and 441, 492; 24 246, 260
// and 583, 500; MXFP4: 24 195, 246 and 439, 501; 32 243, 250 and 525, 525).
inline bool crowded(const fp4_weights* gu, int64_t n) {
  return n > (gu->format == FP4_FORMAT_NVFP4 ? 20 : 32) * gu->experts;
}

// Few enough assignments that the down projection joins them itself (32: 49 us
// with 64 experts and 62 with 128, by streams and a join 48 and 69; 96: 138 and 79).
inline bool few(const fp4_weights* dn, int64_t tokens, int64_t n) {
  return tokens <= 16 && n <= kFewMost && stream_fits(dn);
}

struct ExpertsPlan {
  int64_t tokens;                        // of a slice
  int64_t n;                             // its assignments
  bool inline_rows;                      // sorted by every workgroup for itself
  size_t h, y, off, order, bytes;        // places in the workspace
};

inline ExpertsPlan experts_plan(const fp4_weights* gu, const fp4_weights* dn, int64_t tokens,
                                int64_t top_k) {
  ExpertsPlan p;
  const int64_t most = kSliceBytes / (2 * top_k * dn->cols);
  p.tokens = tokens < most ? tokens : most;
  p.n = p.tokens * top_k;
  p.inline_rows = p.n <= kInlineMost && (!crowded(gu, p.n) || few(dn, p.tokens, p.n));
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t o = at;
    at += (bytes + 255) & ~(size_t)255;
    return o;
  };
  p.h = take((size_t)p.n * dn->cols * 2);
  p.y = take((size_t)p.n * dn->rows * 4);
  p.off = take(p.inline_rows ? 0 : (size_t)(gu->experts + 1) * 4);
  p.order = take(p.inline_rows ? 0 : (size_t)p.n * 4);
  p.bytes = at;
  return p;
}

inline int check_experts(const fp4_weights* gu, const fp4_weights* dn, int64_t tokens,
                         int64_t top_k) {
  if (int rc = check_weights(gu)) return rc;
  if (int rc = check_weights(dn)) return rc;
  if (gu->experts != dn->experts || gu->experts < 1 || gu->experts > 1024 ||
      gu->rows != 2 * dn->cols || gu->cols != dn->rows || gu->cols == 0 || dn->cols == 0)
    return FP4_E_SHAPE;
  if (tokens < 0 || tokens >= ((int64_t)1 << 31) || top_k < 1 || top_k > 64) return FP4_E_SHAPE;
  return FP4_OK;
}

inline hipError_t experts_slice(const fp4_weights* gate_up, const fp4_weights* down,
                                const ExpertsPlan& p, const uint16_t* x, int64_t x_stride,
                                int64_t tokens, const float* weights, const int32_t* experts,
                                int top_k, uint16_t* out, int64_t out_stride, uint8_t* ws,
                                hipStream_t st) {
  const int e = (int)gate_up->experts, inner = (int)down->cols;
  const int64_t n = tokens * top_k;
  ColsArgs a = {};
  a.w = weight_view(gate_up);
  a.x = x;
  a.out = ws + p.h;
  a.xs = x_stride;
  a.os = inner;
  a.tokens = tokens;
  a.ids = experts;
  a.off = (const int32_t*)(ws + p.off);
  a.order = (const int32_t*)(ws + p.order);
  a.top_k = top_k;
  a.experts = e;
  a.inner = inner;
  a.out_vec = 1;
  a.x_per_token = 1;
  ColsArgs b = a;
  b.w = weight_view(down);
  b.x = (const uint16_t*)(ws + p.h);
  b.out = ws + p.y;
  b.xs = inner;
  b.os = down->rows;
  b.out_f32 = 1;
  b.x_per_token = 0;
  a.x_bytes = ((tokens - 1) * x_stride + gate_up->cols) * 2;
  b.x_bytes = n * inner * 2;
  // workgroups' experts: those that have assignments (inline_expert), of one token its
  // assignments themselves, of which there may be more than experts
  const int64_t slots = p.inline_rows && (n < e || tokens == 1) ? n : e;
  const int64_t quads = tokens * (down->rows / 4);
  if (cdiv(quads, kJoinThreads) >= ((int64_t)1 << 31)) return hipErrorInvalidConfiguration;
  hipError_t err = hipSuccess;
  if (!p.inline_rows)
    err = launch(expert_plan_kernel, (unsigned)e, kPlanThreads, st, experts, (int)n, e,
                 (int32_t*)(ws + p.off), (int32_t*)(ws + p.order));
  if (p.inline_rows && few(down, tokens, n)) {
    if (stream_fits(gate_up))
      err = launch_stream<true, kInline>(gate_up->format, a, slots, slots < e ? slots : e, tokens, st);
    else
      err = launch_cols<1, true, kInline>(gate_up->format, a, slots, st);
    b.out = out;
    b.os = out_stride;
    const unsigned grid = (unsigned)cdiv(b.w.rows, 16);
    return first(err, down->format == FP4_FORMAT_NVFP4
                          ? launch(fp4_down_few_kernel<0>, grid, kFewThreads, st, b, weights)
                          : launch(fp4_down_few_kernel<1>, grid, kFewThreads, st, b, weights));
  }
  auto both = [&](auto src) {
    constexpr int S = decltype(src)::value;
    const int64_t busy = slots < e ? slots : e;      // experts that can have tokens
    err = first(err, stream_fits(gate_up)
                         ? launch_stream<true, S>(gate_up->format, a, slots, busy, tokens, st)
                         : launch_cols<1, true, S>(gate_up->format, a, slots, st));
    err = first(err, stream_fits(down)
                         ? launch_stream<false, S>(down->format, b, slots, busy, tokens, st)
                         : launch_cols<2, false, S>(down->format, b, slots, st));
  };
  if (!p.inline_rows && crowded(gate_up, n)) {
    TiledArgs ta = tiled_args(a), tb = tiled_args(b);
    ta.tiles_t = tb.tiles_t = (uint32_t)(n / kTileTokens + e);
    ta.out_vec = tb.out_vec = 1;
    err = first(err, launch_tiled<true, true>(gate_up->format, ta, st));
    err = first(err, launch_tiled<false, true>(down->format, tb, st));
  } else if (p.inline_rows) {
    both(std::integral_constant<int, kInline>{});
  } else {
    both(std::integral_constant<int, kPlanned>{});
  }
  return first(err, launch(experts_join_kernel, (unsigned)cdiv(quads, kJoinThreads), kJoinThreads, st,
                           (const float*)(ws + p.y), weights, experts, tokens, top_k, e,
                           (int)down->rows, out, out_stride));
}

// ------------------------------------------------------------------ routing
inline int check_route(const fp4_routing* r) {
  if (!r) return FP4_E_NULL;
  if (r->tokens < 0 || r->tokens >= ((int64_t)1 << 31) || r->experts < 1 || r->experts > 1024 ||
      r->top_k < 1 || r->top_k > 64 || r->top_k > r->experts)
    return FP4_E_SHAPE;
  if (int rc = check_rows(r->tokens, r->stride, r->experts, 1)) return rc;
  if (!std::isfinite(r->scale)) return FP4_E_SHAPE;
  if (r->tokens > 0 && !r->logits) return FP4_E_NULL;
  return aligned(r->logits, r->logits_bf16 ? 2 : 4) ? FP4_OK : FP4_E_ALIGN;
}

inline int check_choice(const fp4_routing* r) {
  if (r->groups < 1 || r->groups > 64 || r->experts % r->groups || r->top_groups < 1 ||
      r->top_groups > r->groups || r->group_top < 1 || r->group_top > 2 ||
      r->experts / r->groups * r->top_groups < r->top_k)
    return FP4_E_SHAPE;
  return aligned(r->bias, 4) ? FP4_OK : FP4_E_ALIGN;
}

inline RouteArgs route_args(const fp4_routing* r) {
  RouteArgs a;
  a.logits = r->logits;
  a.bias = r->bias;
  a.stride = r->stride;
  a.tokens = r->tokens;
  a.experts = r->experts;
  a.top_k = r->top_k;
  a.groups = r->top_groups < r->groups ? r->groups : 1;      // all groups stay: none to choose
  a.top_groups = r->top_groups;
  a.group_top = r->group_top;
  a.renormalize = r->renormalize;
  a.sigmoid = r->sigmoid != 0;
  a.scale = r->scale;
  return a;
}

// n tokens from the t-th on.
inline RouteArgs route_slice(RouteArgs a, const fp4_routing* r, int64_t t, int64_t n) {
  a.logits = (const uint8_t*)a.logits + t * a.stride * (r->logits_bf16 ? 2 : 4);
  a.tokens = n;
  return a;
}

// Sixteen lanes a token where they hold its experts, 16 each, and its choices and
// one more.
inline bool route_narrow(const RouteArgs& a) { return a.experts <= 256 && a.top_k <= 15; }

// Experts of a lane, so that a group is a run of 2^i lanes; false if none fits.
inline bool route_lanes(RouteArgs& a, int lanes, int most) {
  a.per_lane = most;
  a.group_lanes = 1;
  if (a.groups <= 1) return true;
  const int per = a.experts / a.groups;
  for (int run = 1; run * a.groups <= lanes && per % run == 0; run *= 2)
    if (per / run <= most) {
      a.per_lane = per / run;
      a.group_lanes = run;
      return true;
    }
  return false;
}

// f(lanes a token, values a lane) as compile-time constants.
template <typename F>
hipError_t route_variant(const RouteArgs& a, F&& f) {
  using std::integral_constant;
  if (route_narrow(a)) {
    const integral_constant<int, 16> l;
    if (a.experts <= 64) return f(l, integral_constant<int, 4>{});
    if (a.experts <= 128) return f(l, integral_constant<int, 8>{});
    return f(l, integral_constant<int, 16>{});
  }
  const integral_constant<int, 64> l;
  if (a.experts <= 256) return f(l, integral_constant<int, 4>{});
  return f(l, integral_constant<int, 16>{});
}

// ------------------------------------------------------------------ norms around a block
inline int check_residual(const fp4_residual* a) {
  if (!a) return FP4_E_NULL;
  if (a->tokens < 0 || a->tokens >= ((int64_t)1 << 31) || a->dim < 8 || a->dim > 16384 ||
      a->dim % 8)
    return FP4_E_SHAPE;
  if (!(a->eps >= 0.0f) || std::isinf(a->eps) || !std::isfinite(a->scale)) return FP4_E_SHAPE;
  if (!a->weight) return FP4_E_NULL;
  if (!aligned(a->weight, 16) || !aligned(a->block_weight, 16) ||
      !aligned(a->gate, a->token_gate ? 2 : 16))
    return FP4_E_ALIGN;
  return FP4_OK;
}

inline int check_residual_pair(const fp4_residual* a, const void* p, int64_t ps, const void* q,
                               int64_t qs) {
  if (a->tokens == 0) return FP4_OK;
  if (!p || !q) return FP4_E_NULL;
  if (int rc = check_rows(a->tokens, ps, a->dim, 8)) return rc;
  if (int rc = check_rows(a->tokens, qs, a->dim, 8)) return rc;
  return aligned(p, 16) && aligned(q, 16) ? FP4_OK : FP4_E_ALIGN;
}

inline ResidualArgs residual_args(const fp4_residual* a) {
  ResidualArgs r;
  r.x = a->x;
  r.b = a->block;
  r.bw = a->block_weight;
  r.w = a->weight;
  r.gate = a->gate;
  r.xs = a->x_stride;
  r.bs = a->block_stride;
  r.tokens = a->tokens;
  r.dim = a->dim;
  r.token_gate = a->token_gate != 0;
  r.scale = a->scale;
  r.eps = a->eps;
  return r;
}

// f(waves a row, chunks a thread).
template <typename F>
hipError_t residual_variant(int dim, F&& f) {
  using std::integral_constant;
  if (dim <= 512) return f(integral_constant<int, 1>{}, integral_constant<int, 1>{});
  if (dim <= 1024) return f(integral_constant<int, 1>{}, integral_constant<int, 2>{});
  if (dim <= 2048) return f(integral_constant<int, 4>{}, integral_constant<int, 1>{});
  if (dim <= 4096) return f(integral_constant<int, 4>{}, integral_constant<int, 2>{});
  if (dim <= 8192) return f(integral_constant<int, 16>{}, integral_constant<int, 1>{});
  return f(integral_constant<int, 16>{}, integral_constant<int, 2>{});
}

inline int64_t residual_groups(int64_t tokens, int dim) {
  const int64_t g = dim <= 1024 ? cdiv(tokens, RowShape<1>::kRows) : tokens;
  return g < kResidualMaxGroups ? g : kResidualMaxGroups;
}

}  // namespace feedforward
}  // namespace fp4q

extern "C" {

size_t fp4_linear_workspace_bytes(const fp4_weights*, int64_t) { return 0; }

int fp4_linear(const fp4_weights* w, const uint16_t* x, int64_t x_stride, int64_t tokens, void* out,
               int64_t out_stride, int out_f32, void* ws, size_t ws_bytes, void* stream) {
  using namespace fp4q;
  using namespace fp4q::feedforward;
  if (int rc = check_weights(w)) return rc;
  if (w->experts != 1 || tokens < 0 || tokens >= ((int64_t)1 << 31)) return FP4_E_SHAPE;
  if (tokens == 0 || w->rows == 0) return FP4_OK;
  if ((!x && w->cols) || !out) return FP4_E_NULL;
  if (int rc = check_rows(tokens, x_stride, w->cols, 8)) return rc;
  if (x_stride >= kMaxXStride) return FP4_E_SHAPE;
  if (int rc = check_rows(tokens, out_stride, w->rows, 1)) return rc;
  if (!aligned(x, 16) || !aligned(out, out_f32 ? 4 : 2)) return FP4_E_ALIGN;
  const int64_t most = linear_slice(w->rows);
  hipError_t err = hipSuccess;
  for (int64_t t = 0; t < tokens && err == hipSuccess; t += most)
    err = linear_call(w, x + t * x_stride, x_stride, tokens - t < most ? tokens - t : most,
                      (uint8_t*)out + t * out_stride * (out_f32 ? 4 : 2), out_stride, out_f32 != 0,
                      (hipStream_t)stream);
  return launched(err);
}

int expert_route(const fp4_routing* r, float* weights, int32_t* experts, void* stream) {
  using namespace fp4q;
  using namespace fp4q::feedforward;
  if (int rc = check_route(r)) return rc;
  if (int rc = check_choice(r)) return rc;
  if (r->tokens == 0) return FP4_OK;
  if (!weights || !experts) return FP4_E_NULL;
  if (!aligned(weights, 4) || !aligned(experts, 4)) return FP4_E_ALIGN;
  RouteArgs a = route_args(r);
  return launched(route_variant(a, [&](auto lpt, auto v) {
    constexpr int L = decltype(lpt)::value, V = decltype(v)::value, V64 = (L * V + 63) / 64;
    auto go = [&](auto kernel, int tokens) {
      return in_slices(r->tokens, kRouteWaves * tokens, kRouteThreads, [&](int64_t t, int64_t n) {
        return launch(kernel, (unsigned)cdiv(n, kRouteWaves * tokens), kRouteThreads,
                      (hipStream_t)stream, route_slice(a, r, t, n), weights + t * a.top_k,
                      experts + t * a.top_k);
      });
    };
    if (!route_lanes(a, L, V) || a.top_k >= L)
      return r->logits_bf16 ? go(expert_route64_kernel<V64, true>, 1)
                            : go(expert_route64_kernel<V64, false>, 1);
    return r->logits_bf16 ? go(expert_route_kernel<L, V, true>, 64 / L)
                          : go(expert_route_kernel<L, V, false>, 64 / L);
  }));
}

int expert_route_backward(const fp4_routing* r, const float* dweights, const int32_t* experts,
                          void* dlogits, int64_t dlogits_stride, void* stream) {
  using namespace fp4q;
  using namespace fp4q::feedforward;
  if (int rc = check_route(r)) return rc;
  if (int rc = check_rows(r->tokens, dlogits_stride, r->experts, 1)) return rc;
  if (r->tokens == 0) return FP4_OK;
  if (!dweights || !experts || !dlogits) return FP4_E_NULL;
  if (!aligned(dweights, 4) || !aligned(experts, 4) || !aligned(dlogits, r->logits_bf16 ? 2 : 4))
    return FP4_E_ALIGN;
  RouteArgs a = route_args(r);
  a.bias = nullptr;
  return launched(route_variant(a, [&](auto lpt, auto v) {
    constexpr int L = decltype(lpt)::value, V = decltype(v)::value;
    auto go = [&](auto kernel) {
      constexpr int G = kRouteWaves * (64 / L);
      return in_slices(r->tokens, G, kRouteThreads, [&](int64_t t, int64_t n) {
        return launch(kernel, (unsigned)cdiv(n, G), kRouteThreads, (hipStream_t)stream,
                      route_slice(a, r, t, n), dweights + t * a.top_k, experts + t * a.top_k,
                      (uint8_t*)dlogits + t * dlogits_stride * (r->logits_bf16 ? 2 : 4),
                      dlogits_stride);
      });
    };
    return r->logits_bf16 ? go(expert_route_backward_kernel<L, V, true>)
                          : go(expert_route_backward_kernel<L, V, false>);
  }));
}

size_t fp4_experts_workspace_bytes(const fp4_weights* gate_up, const fp4_weights* down,
                                   int64_t tokens, int64_t top_k) {
  using namespace fp4q::feedforward;
  if (check_experts(gate_up, down, tokens, top_k) || tokens == 0) return 0;
  return experts_plan(gate_up, down, tokens, top_k).bytes;
}

int fp4_experts(const fp4_weights* gate_up, const fp4_weights* down, const uint16_t* x,
                int64_t x_stride, int64_t tokens, const float* weights, const int32_t* experts,
                int64_t top_k, uint16_t* out, int64_t out_stride, void* ws, size_t ws_bytes,
                void* stream) {
  using namespace fp4q;
  using namespace fp4q::feedforward;
  if (int rc = check_experts(gate_up, down, tokens, top_k)) return rc;
  if (tokens == 0) return FP4_OK;
  if (!x || !weights || !experts || !out || !ws) return FP4_E_NULL;
  if (int rc = check_rows(tokens, x_stride, gate_up->cols, 8)) return rc;
  if (x_stride >= kMaxXStride) return FP4_E_SHAPE;
  if (int rc = check_rows(tokens, out_stride, gate_up->cols, 8)) return rc;
  if (!aligned(x, 16) || !aligned(out, 16) || !aligned(weights, 4) || !aligned(experts, 4) ||
      !aligned(ws, 16))
    return FP4_E_ALIGN;
  const ExpertsPlan p = experts_plan(gate_up, down, tokens, top_k);
  if (ws_bytes < p.bytes) return FP4_E_WORKSPACE;
  // rows of x in reach of 31 bits
  int64_t most = (kSliceBytes / 2 - gate_up->cols) / x_stride + 1;
  most = most < p.tokens ? most : p.tokens;
  hipError_t err = hipSuccess;
  for (int64_t t = 0; t < tokens && err == hipSuccess; t += most)
    err = experts_slice(gate_up, down, p, x + t * x_stride, x_stride,
                        tokens - t < most ? tokens - t : most, weights + t * top_k,
                        experts + t * top_k, (int)top_k, out + t * out_stride, out_stride,
                        (uint8_t*)ws, (hipStream_t)stream);
  return launched(err);
}

int residual_norm(const fp4_residual* a, uint16_t* y, int64_t y_stride, uint16_t* z,
                  int64_t z_stride, void* stream) {
  using namespace fp4q;
  using namespace fp4q::feedforward;
  if (int rc = check_residual(a)) return rc;
  if (int rc = check_residual_pair(a, a->x, a->x_stride, a->block, a->block_stride)) return rc;
  if (int rc = check_residual_pair(a, y, y_stride, z, z_stride)) return rc;
  if (a->tokens == 0) return FP4_OK;
  const ResidualArgs r = residual_args(a);
  return launched(residual_variant(a->dim, [&](auto wpr, auto ch) {
    constexpr int W = decltype(wpr)::value, CH = decltype(ch)::value;
    using S = RowShape<W>;
    return in_slices(r.tokens, S::kRows, S::kAll, [&](int64_t t, int64_t n) {
      ResidualArgs part = r;
      part.x += t * r.xs;
      part.b += t * r.bs;
      if (r.gate && r.token_gate) part.gate += t;
      part.tokens = n;
      return launch(residual_norm_kernel<W, CH>, (unsigned)cdiv(n, S::kRows), S::kAll,
                    (hipStream_t)stream, part, y + t * y_stride, y_stride, z + t * z_stride, z_stride);
    });
  }));
}

size_t residual_norm_workspace_bytes(int64_t tokens, int dim) {
  if (tokens < 0 || dim < 8 || dim > 16384) return 0;
  return (size_t)fp4q::feedforward::residual_groups(tokens, dim) * 2 * (size_t)dim * sizeof(float);
}

int residual_norm_backward(const fp4_residual* a, const uint16_t* dy, int64_t dy_stride,
                           const uint16_t* dz, int64_t dz_stride, uint16_t* dx, int64_t dx_stride,
                           uint16_t* dblock, int64_t dblock_stride, float* dblock_weight,
                           float* dweight, float* dgate, void* ws, size_t ws_bytes, void* stream) {
  using namespace fp4q;
  using namespace fp4q::feedforward;
  if (int rc = check_residual(a)) return rc;
  if (int rc = check_residual_pair(a, a->x, a->x_stride, a->block, a->block_stride)) return rc;
  if (int rc = check_residual_pair(a, dy, dy_stride, dz, dz_stride)) return rc;
  if (int rc = check_residual_pair(a, dx, dx_stride, dblock, dblock_stride)) return rc;
  if ((dblock_weight && !a->block_weight) || (dgate && !a->gate)) return FP4_E_NULL;
  const ResidualArgs r = residual_args(a);
  const bool channel = a->gate && !a->token_gate;
  const bool sums = dblock_weight || dweight || (dgate && channel);
  if (!aligned(dblock_weight, 4) || !aligned(dweight, 4) || !aligned(dgate, 4) || !aligned(ws, 16))
    return FP4_E_ALIGN;
  const size_t need = residual_norm_workspace_bytes(a->tokens, a->dim);
  if (sums && need > 0 && !ws) return FP4_E_NULL;
  if (sums && ws_bytes < need) return FP4_E_WORKSPACE;
  hipStream_t st = (hipStream_t)stream;
  const int64_t groups = residual_groups(a->tokens, a->dim);
  hipError_t e = hipSuccess;
  if (groups > 0)
    e = residual_variant(a->dim, [&](auto wpr, auto ch) {
      constexpr int W = decltype(wpr)::value, CH = decltype(ch)::value;
      return launch(residual_norm_bwd_kernel<W, CH>, (unsigned)groups, RowShape<W>::kAll, st, r, dy,
                    dy_stride, dz, dz_stride, dx, dx_stride, dblock, dblock_stride,
                    sums ? (float*)ws : nullptr, dgate);
    });
  if (sums)
    e = first(e, launch(residual_norm_dw_kernel, (unsigned)cdiv(2 * (int64_t)a->dim, kResidualDwCols),
                        kResidualDwCols * kResidualDwRows, st, (const float*)ws, (int)groups, r,
                        dblock_weight, dweight, dgate));
  return launched(e);
}

}  // extern "C"
