// kv_common.h -- layout of the paged FP4 key/value cache, and the bf16 stores of
// the operators around it.
//
// Page size P (a power of two, 16 at least), H kv heads, D values per head,
// G values per scale (NVFP4 16, MXFP4 32); [page][head] outermost:
//   k_codes  [P][D/2]     k_scales [P][D/G]     a token's key is one run
//   v_codes  [D/2][P]     v_scales [D/G][P]     a channel pair's tokens are one run
// The two operands of attention contract over different axes (keys over
// channels, values over tokens); with each stored along its own, a lane's
// load is a run of the axis that its matrix operand contracts over, and
// neither needs a transpose on the way in.
#pragma once

#include "device_common.h"

namespace fp4q {

struct KvView {
  uint8_t *kc, *ks, *vc, *vs;
  const float *kam, *vam;                // [heads] (NVFP4)
  int64_t pages;
  int page_shift, heads, dim;
};

// Nearest-even bf16 pair (lo, hi).
__device__ __forceinline__ uint32_t bf16x2_of(float lo, float hi) {
  typedef __bf16 bf16x2_v __attribute__((ext_vector_type(2)));
  bf16x2_v v;
  v[0] = (__bf16)lo;
  v[1] = (__bf16)hi;
  return __builtin_bit_cast(uint32_t, v);
}

__device__ __forceinline__ uint4 pack8(const float* y) {
  return make_uint4(bf16x2_of(y[0], y[1]), bf16x2_of(y[2], y[3]), bf16x2_of(y[4], y[5]),
                    bf16x2_of(y[6], y[7]));
}

// Page of a slot, or -1 where there is none.
__device__ __forceinline__ int64_t slot_page(const KvView& c, int64_t slot) {
  const int64_t page = slot >> c.page_shift;
  return slot >= 0 && page < c.pages ? page : -1;
}

}  // namespace fp4q
