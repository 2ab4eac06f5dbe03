// attention.hip -- entry points of the norm with rotation and of attention
// over the paged FP4 cache: argument checks on the host, then kernel
// launches on the caller's stream.  See include/fp4q.h for the contract.
#include <hip/hip_runtime.h>

#include <cmath>

#include "host_common.h"
#include "kv_attention_kernels.h"
#include "kv_host.h"
#include "kv_tiled_kernels.h"
#include "rope_kernels.h"

using namespace fp4q;

namespace {

// ------------------------------------------------------------------ norm + rotation
// Lanes per head: D / 8 rounded up to a power of two.
int lanes_per_head(int dim) {
  int l = 1;
  while (l * 8 < dim) l *= 2;
  return l;
}

int check_tokens(int64_t tokens, int64_t stride, int64_t width) {
  if (stride < width || stride % 8 || stride >= kMaxElems) return FP4_E_SHAPE;
  if (tokens > 0 && stride > kMaxElems / tokens) return FP4_E_SHAPE;
  return FP4_OK;
}

int check_rope(const fp4_qk_rope* a) {
  if (!a) return FP4_E_NULL;
  if (a->tokens < 0 || a->tokens >= ((int64_t)1 << 31) || a->q_heads < 0 || a->k_heads < 0 ||
      a->q_heads > 65536 || a->k_heads > 65536)
    return FP4_E_SHAPE;
  if (a->head_dim < 16 || a->head_dim > 256 || a->head_dim % 8) return FP4_E_SHAPE;
  if (a->rot_dim < 0 || a->rot_dim > a->head_dim || a->rot_dim % 16 || a->table_rows < 0)
    return FP4_E_SHAPE;
  if (a->flags & ~(uint32_t)FP4_ROPE_INTERLEAVED) return FP4_E_FLAGS;
  if (!(a->eps >= 0.0f) || std::isinf(a->eps)) return FP4_E_SHAPE;
  if (a->tokens == 0 || a->q_heads + a->k_heads == 0) return FP4_OK;
  if ((a->q_heads && !a->q) || (a->k_heads && !a->k)) return FP4_E_NULL;
  if (a->rot_dim > 0 && (!a->positions || !a->table)) return FP4_E_NULL;
  if (a->rot_dim > 0 && a->table_rows == 0) return FP4_E_SHAPE;
  if (a->q_heads)
    if (int rc = check_tokens(a->tokens, a->q_stride, (int64_t)a->q_heads * a->head_dim)) return rc;
  if (a->k_heads)
    if (int rc = check_tokens(a->tokens, a->k_stride, (int64_t)a->k_heads * a->head_dim)) return rc;
  if (!aligned(a->q, 16) || !aligned(a->k, 16) || !aligned(a->q_weight, 16) ||
      !aligned(a->k_weight, 16) || !aligned(a->positions, 8) || !aligned(a->table, 16))
    return FP4_E_ALIGN;
  return FP4_OK;
}

// A second tensor of the same heads (outputs and gradients).
int check_rope_pair(const fp4_qk_rope* a, const void* q, int64_t qs, const void* k, int64_t ks) {
  if (a->tokens == 0) return FP4_OK;
  if ((a->q_heads && !q) || (a->k_heads && !k)) return FP4_E_NULL;
  if (a->q_heads)
    if (int rc = check_tokens(a->tokens, qs, (int64_t)a->q_heads * a->head_dim)) return rc;
  if (a->k_heads)
    if (int rc = check_tokens(a->tokens, ks, (int64_t)a->k_heads * a->head_dim)) return rc;
  return aligned(q, 16) && aligned(k, 16) ? FP4_OK : FP4_E_ALIGN;
}

RopeArgs rope_args(const fp4_qk_rope* a) {
  RopeArgs r;
  r.q = a->q;
  r.k = a->k;
  r.qw = a->q_weight;
  r.kw = a->k_weight;
  r.pos = a->positions;
  r.table = a->table;
  r.qs = a->q_stride;
  r.ks = a->k_stride;
  r.tokens = a->tokens;
  r.table_rows = a->table_rows;
  r.hq = a->q_heads;
  r.hk = a->k_heads;
  r.dim = a->head_dim;
  r.rot = a->rot_dim;
  r.eps = a->eps;
  // heads per lane group: more share one read of the token's cosines, fewer
  // keep every CU supplied with small calls
  const int64_t heads = a->q_heads + a->k_heads;
  const int64_t groups = (int64_t)num_cus() * 8 * (64 / lanes_per_head(a->head_dim));
  const int64_t hpg = heads ? a->tokens * heads / groups : 1;
  r.hpg = (int)(hpg < 1 ? 1 : (hpg > 8 ? 8 : hpg));
  r.chunks = (int)cdiv(heads, r.hpg);
  return r;
}

// f(lanes per head, interleaved) with both as compile-time constants.
template <typename F>
hipError_t rope_variant(const fp4_qk_rope* a, F&& f) {
  const bool inter = a->flags & FP4_ROPE_INTERLEAVED;
  auto pick = [&](auto lph) {
    return inter ? f(lph, std::true_type{}) : f(lph, std::false_type{});
  };
  switch (lanes_per_head(a->head_dim)) {
    case 2: return pick(std::integral_constant<int, 2>{});
    case 4: return pick(std::integral_constant<int, 4>{});
    case 8: return pick(std::integral_constant<int, 8>{});
    case 16: return pick(std::integral_constant<int, 16>{});
    default: return pick(std::integral_constant<int, 32>{});
  }
}

// Workgroups of the backward pass: the rows of partial weight gradients, which
// a second launch joins; one writes the gradients itself.
constexpr int kRopeAlone = 4;
int64_t rope_bwd_groups(const fp4_qk_rope* a, const RopeArgs& r) {
  const int64_t per = kRopeThreads / lanes_per_head(a->head_dim);
  const int64_t g = cdiv(a->tokens * r.chunks, per);
  // a few rounds of one workgroup cost less than the second launch that joins
  // several (40 heads of 128 of one token, forward and backward: 13.0 us, two
  // launches 15.3; 4 tokens in 10 rounds: 21.1 and 15.3)
  if (g <= kRopeAlone) return 1;
  return g < kRopeMaxGroups ? g : kRopeMaxGroups;
}

// ------------------------------------------------------------------ attention
constexpr int64_t kMaxRows = ((int64_t)1 << 31) - 1;   // query rows: the kernels count them in 32 bits

int check_attention_sizes(const fp4_kv_cache* c, const fp4_kv_queries* x) {
  if (!x) return FP4_E_NULL;
  if (int rc = check_kv_cache(c)) return rc;
  if (x->tokens < 0 || x->tokens >= ((int64_t)1 << 31) || x->seqs < 0 ||
      x->seqs >= ((int64_t)1 << 31) || x->table_width < 0 || x->max_q < 0 ||
      x->table_width > (((int64_t)1 << 31) - 1) / c->page_size)
    return FP4_E_SHAPE;
  if (x->q_heads < 1 || x->q_heads > 65536 || x->q_heads % c->heads) return FP4_E_SHAPE;
  if (x->tokens > kMaxRows / x->q_heads || x->seqs > kMaxRows / x->q_heads) return FP4_E_SHAPE;
  if (!x->cu_q && x->tokens != x->seqs) return FP4_E_SHAPE;
  if (x->window < 0 || !(x->softcap >= 0.0f) || std::isinf(x->softcap) || !std::isfinite(x->scale))
    return FP4_E_SHAPE;
  return x->tokens > 0 && x->seqs == 0 ? FP4_E_SHAPE : FP4_OK;
}

int check_attention(const fp4_kv_cache* c, const fp4_kv_queries* x, const uint16_t* out,
                    int64_t out_stride, const float* lse) {
  if (int rc = check_attention_sizes(c, x)) return rc;
  if (x->tokens == 0) return FP4_OK;
  if (!x->q || !out || !x->kv_lens || (x->table_width > 0 && !x->page_table)) return FP4_E_NULL;
  const int64_t width = (int64_t)x->q_heads * c->head_dim;
  if (int rc = check_tokens(x->tokens, x->q_stride, width)) return rc;
  if (int rc = check_tokens(x->tokens, out_stride, width)) return rc;
  if (!aligned(x->q, 16) || !aligned(out, 16) || !aligned(x->page_table, 4) ||
      !aligned(x->kv_lens, 4) || !aligned(x->cu_q, 4) || !aligned(lse, 4))
    return FP4_E_ALIGN;
  return FP4_OK;
}

// How a call is cut up: columns of 16 rows per tile (0: the tiled kernel),
// tiles of the grid (an upper bound of what the sequences need), parts of the
// context.
struct AttnPlan {
  int nt;
  bool wide;                             // a block of keys lies in one page
  int64_t tiles, splits, want, places;
};

AttnPlan attention_plan(const fp4_kv_cache* c, const fp4_kv_queries* x) {
  AttnPlan p;
  const int64_t group = x->q_heads / c->heads;
  const int64_t known = x->max_q < x->tokens ? x->max_q : x->tokens;
  const int64_t most = !x->cu_q ? 1 : (known > 0 ? known : cdiv(x->tokens, x->seqs));
  const int64_t rows = most * group;
  p.nt = rows <= 16 ? 1 : (rows <= 32 && c->head_dim < 256 ? 2 : 0);
  const int64_t m = p.nt ? 16 * p.nt : kTileRows;
  p.tiles = x->cu_q ? x->tokens * group / m + x->seqs : x->seqs * cdiv(group, m);
  // keys in reach of a tile, at most
  int64_t keys = x->table_width * c->page_size;
  const int64_t span = most < m / group + 2 ? most : m / group + 2;    // new tokens of a tile
  if (x->window > 0 && keys > x->window + span) keys = x->window + span;
  const int64_t blocks = cdiv(keys, kAttnKeys);
  // Workgroups wanted per kv head.  How they are shared out among the
  // sequences depends on lengths that only the device knows (item_of); a
  // tile gets at most four times an even share.  As many as run at once, so
  // that all of them end together: chunks of 512 tokens over 6144 cached, heads
  // of 128, 3 to a CU: 139 us, 2: 161, 4: 162, 6: 166.  (Two column tiles of
  // heads of 64 would run 3 by their registers and are counted as 2.)
  p.wide = c->page_size >= (p.nt == 0 ? kTileKeys : kAttnKeys);
  const int d = c->head_dim;
  const int per_cu = p.nt == 0 ? tile_waves(d, p.wide, x->softcap > kShortCap)
                               : (p.nt == 2 || d == 256 ? 2 : (d == 128 ? 3 : 4));
  p.want = cdiv(per_cu * (int64_t)num_cus(), c->heads);
  // One part, without the launch that joins several, as long as a wave has two
  // blocks at most: a context of 512 tokens 7.8 us (parts 9.4), of 768 9.4
  // (9.4), of 1024 10.9 (9.7).
  const int64_t share = cdiv(4 * p.want, p.tiles);
  const int64_t room = p.nt && blocks <= 8 ? 1 : cdiv(blocks, 4);
  p.splits = p.tiles >= p.want ? 1 : (share < room ? share : room);
  p.splits = p.splits < 1 ? 1 : (p.splits > 64 ? 64 : p.splits);
  // every tile has one part and the rest come to a.want together
  p.places = p.tiles + (p.splits > 1 ? p.want : 0);
  return p;
}

size_t attention_ws(const fp4_kv_cache* c, const fp4_kv_queries* x, const AttnPlan& p) {
  if (p.splits <= 1) return 0;
  return (size_t)p.splits * x->tokens * x->q_heads * (c->head_dim + 2) * sizeof(float) +
         (size_t)x->tokens * x->q_heads * sizeof(int);
}

template <int MODE, int D>
hipError_t launch_attention(const AttnPlan& p, const AttnArgs& a, hipStream_t st) {
  const unsigned grid = (unsigned)(p.places * a.c.heads);
  hipError_t e = hipSuccess;
  if (p.nt == 0) {
    auto go = [&](auto cap) {
      constexpr bool LONG = decltype(cap)::value;
      return p.wide ? launch(kv_tiled_kernel<MODE, D, true, LONG>, grid, kThreads, st, a)
                    : launch(kv_tiled_kernel<MODE, D, false, LONG>, grid, kThreads, st, a);
    };
    e = a.cap > kShortCap ? go(std::true_type{}) : go(std::false_type{});
  } else {
    auto go = [&](auto nt) {
      constexpr int N = decltype(nt)::value;
      return p.wide ? launch(kv_attention_kernel<MODE, D, N, 4, true>, grid, 256, st, a)
                    : launch(kv_attention_kernel<MODE, D, N, 4, false>, grid, 256, st, a);
    };
    if (p.nt == 1) e = go(std::integral_constant<int, 1>{});
    else if constexpr (D < 256) e = go(std::integral_constant<int, 2>{});
  }
  if (p.splits > 1) {
    // as many lanes on a row's parts as leave a lane 4 of the even share
    const int lanes = D / 4, most = kThreads / lanes;
    const int64_t share = cdiv(p.want, p.tiles), parts = share < p.splits ? share : p.splits;
    int groups = 1;
    while (groups < most && groups * 4 < parts) groups *= 2;
    e = first(e, launch(kv_attention_join_kernel<MODE, D>,
                        (unsigned)cdiv(a.tokens * a.hq, kThreads / (lanes * groups)), kThreads, st,
                        a, groups, a.tokens * a.hq <= 4096));
  }
  return e;
}

template <int MODE>
hipError_t launch_attention(int dim, const AttnPlan& p, const AttnArgs& a, hipStream_t st) {
  switch (dim) {
    case 64: return launch_attention<MODE, 64>(p, a, st);
    case 128: return launch_attention<MODE, 128>(p, a, st);
    default: return launch_attention<MODE, 256>(p, a, st);
  }
}

}  // namespace

extern "C" {

int qk_norm_rope(const fp4_qk_rope* a, uint16_t* q_out, int64_t q_out_stride, uint16_t* k_out,
                 int64_t k_out_stride, void* stream) {
  if (int rc = check_rope(a)) return rc;
  if (int rc = check_rope_pair(a, q_out, q_out_stride, k_out, k_out_stride)) return rc;
  if (a->tokens == 0 || a->q_heads + a->k_heads == 0) return FP4_OK;
  const RopeArgs r = rope_args(a);
  return launched(rope_variant(a, [&](auto lph, auto inter) {
    constexpr int L = decltype(lph)::value;
    return launch(qk_norm_rope_kernel<L, decltype(inter)::value>,
                  (unsigned)cdiv(r.tokens * r.chunks, kRopeThreads / L), kRopeThreads,
                  (hipStream_t)stream, r, q_out, q_out_stride, k_out, k_out_stride);
  }));
}

size_t qk_norm_rope_workspace_bytes(int head_dim) {
  if (head_dim < 16 || head_dim > 256) return 0;
  return (size_t)kRopeMaxGroups * 2 * (size_t)head_dim * sizeof(float);
}

int qk_norm_rope_backward(const fp4_qk_rope* a, const uint16_t* dq_out, int64_t dq_out_stride,
                          const uint16_t* dk_out, int64_t dk_out_stride, uint16_t* dq,
                          int64_t dq_stride, uint16_t* dk, int64_t dk_stride, float* dq_weight,
                          float* dk_weight, void* ws, size_t ws_bytes, void* stream) {
  if (int rc = check_rope(a)) return rc;
  if (int rc = check_rope_pair(a, dq_out, dq_out_stride, dk_out, dk_out_stride)) return rc;
  if (int rc = check_rope_pair(a, dq, dq_stride, dk, dk_stride)) return rc;
  const bool want_w = dq_weight || dk_weight;
  if ((dq_weight && !a->q_weight) || (dk_weight && !a->k_weight)) return FP4_E_NULL;
  if (want_w && !ws) return FP4_E_NULL;
  if (!aligned(dq_weight, 4) || !aligned(dk_weight, 4) || !aligned(ws, 4)) return FP4_E_ALIGN;
  if (want_w && ws_bytes < qk_norm_rope_workspace_bytes(a->head_dim)) return FP4_E_WORKSPACE;
  const RopeArgs r = rope_args(a);
  const bool none = a->tokens == 0 || a->q_heads + a->k_heads == 0;
  if (none && !want_w) return FP4_OK;
  hipStream_t st = (hipStream_t)stream;
  const int64_t groups = none ? 0 : rope_bwd_groups(a, r);
  hipError_t e = hipSuccess;
  if (!none)
    e = rope_variant(a, [&](auto lph, auto inter) {
      return launch(qk_norm_rope_bwd_kernel<decltype(lph)::value, decltype(inter)::value>,
                    (unsigned)groups, kRopeThreads, st, r, dq_out, dq_out_stride, dk_out,
                    dk_out_stride, dq, dq_stride, dk, dk_stride,
                    want_w && groups > 1 ? (float*)ws : nullptr, dq_weight, dk_weight);
    });
  if (want_w && groups != 1)
    e = first(e, launch(qk_norm_rope_dw_kernel, (unsigned)cdiv(2 * a->head_dim, kDwCols), kDwThreads,
                        st, (const float*)ws, (int)groups, a->head_dim, dq_weight, dk_weight));
  return launched(e);
}

size_t fp4_kv_attention_workspace_bytes(const fp4_kv_cache* cache, const fp4_kv_queries* x) {
  if (check_attention_sizes(cache, x) || x->tokens == 0) return 0;
  return attention_ws(cache, x, attention_plan(cache, x));
}

int fp4_kv_attention(const fp4_kv_cache* c, const fp4_kv_queries* x, uint16_t* out,
                     int64_t out_stride, float* lse, void* ws, size_t ws_bytes, void* stream) {
  if (int rc = check_attention(c, x, out, out_stride, lse)) return rc;
  if (!aligned(ws, 16)) return FP4_E_ALIGN;
  if (x->tokens == 0) return FP4_OK;
  const AttnPlan p = attention_plan(c, x);
  if (p.places > (((int64_t)1 << 32) - 1) / kThreads / c->heads) return FP4_E_SHAPE;
  const size_t need = attention_ws(c, x, p);
  if (need > 0 && !ws) return FP4_E_NULL;
  if (ws_bytes < need) return FP4_E_WORKSPACE;
  AttnArgs a;
  a.c = kv_view(c);
  a.q = x->q;
  a.pt = (const ConstInt*)x->page_table;
  a.lens = (const ConstInt*)x->kv_lens;
  a.cu = (const ConstInt*)x->cu_q;
  a.out = out;
  a.lse = lse;
  a.qs = x->q_stride;
  a.os = out_stride;
  a.tokens = x->tokens;
  a.seqs = x->seqs;
  a.width = x->table_width;
  a.hq = x->q_heads;
  a.group = x->q_heads / c->heads;
  a.window = x->window;
  a.scale = x->scale;
  a.cap = x->softcap;
  a.splits = (int)p.splits;
  a.want = (uint32_t)p.want;
  a.po = (float*)ws;
  const int64_t rows = need ? x->tokens * x->q_heads : 0;
  a.pm = a.po + p.splits * rows * c->head_dim;
  a.parts = (int*)(a.pm + p.splits * rows * 2);
  hipStream_t st = (hipStream_t)stream;
  switch (kv_mode(c)) {
    case 0: return launched(launch_attention<0>(c->head_dim, p, a, st));
    case 1: return launched(launch_attention<1>(c->head_dim, p, a, st));
    default: return launched(launch_attention<2>(c->head_dim, p, a, st));
  }
}

}  // extern "C"
