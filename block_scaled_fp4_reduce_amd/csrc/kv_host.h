// kv_host.h -- host checks of an fp4_kv_cache and its view for the kernels.
#pragma once

#include "host_common.h"
#include "kv_common.h"

namespace fp4q {

// 0 NVFP4, 1 NVFP4 with 4/6, 2 MXFP4 (the kernels' MODE).
inline int kv_mode(const fp4_kv_cache* c) {
  return c->format == FP4_FORMAT_MXFP4 ? 2 : (c->flags & FP4_FOUR_OVER_SIX ? 1 : 0);
}

inline int check_kv_cache(const fp4_kv_cache* c) {
  if (!c) return FP4_E_NULL;
  if (c->format != FP4_FORMAT_NVFP4 && c->format != FP4_FORMAT_MXFP4) return FP4_E_FLAGS;
  const bool nv = c->format == FP4_FORMAT_NVFP4;
  if (c->flags & ~(uint32_t)(nv ? FP4_FOUR_OVER_SIX : 0)) return FP4_E_FLAGS;
  if (c->pages < 0 || c->heads < 1 || c->heads > 65536) return FP4_E_SHAPE;
  if (c->page_size < 16 || c->page_size > 4096 || (c->page_size & (c->page_size - 1)))
    return FP4_E_SHAPE;
  if (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256) return FP4_E_SHAPE;
  if (c->pages >= ((int64_t)1 << 31) ||
      c->pages > kMaxElems / ((int64_t)c->heads * c->page_size * c->head_dim))
    return FP4_E_SHAPE;
  if (c->pages > 0 && (!c->k_codes || !c->k_scales || !c->v_codes || !c->v_scales))
    return FP4_E_NULL;
  if (nv && (!c->k_amax || !c->v_amax)) return FP4_E_NULL;
  if (!aligned(c->k_codes, 16) || !aligned(c->v_codes, 16) || !aligned(c->k_scales, 16) ||
      !aligned(c->v_scales, 16) || !aligned(c->k_amax, 4) || !aligned(c->v_amax, 4))
    return FP4_E_ALIGN;
  return FP4_OK;
}

inline KvView kv_view(const fp4_kv_cache* c) {
  KvView v;
  v.kc = c->k_codes;
  v.ks = c->k_scales;
  v.vc = c->v_codes;
  v.vs = c->v_scales;
  v.kam = c->k_amax;
  v.vam = c->v_amax;
  v.pages = c->pages;
  v.page_shift = __builtin_ctz((unsigned)c->page_size);
  v.heads = c->heads;
  v.dim = c->head_dim;
  return v;
}

}  // namespace fp4q
