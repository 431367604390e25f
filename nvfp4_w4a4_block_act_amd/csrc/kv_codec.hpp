// Device steps of the calibrated FP8 (E4M3) KV-cache codec, shared by the codec's
// own kernels (kv_fp8.hip) and the paged cache's append (kv_append.hip).
#pragma once

#include "common.hpp"

namespace nvfp4 {

__device__ __forceinline__ float kv_g_enc(float amax) { return (amax == 0.0f) ? 0.0f : 448.0f / amax; }

// Codes of one bf16 word pair (elements lo, hi of `w`), as bits 0-15 of the result.
__device__ __forceinline__ uint32_t kv_encode_pair(uint32_t w, float g) {
  const float y0 = __uint_as_float((w << 16) & 0x7FFF0000u) * g;
  const float y1 = __uint_as_float(w & 0x7FFF0000u) * g;
  const uint32_t m = e4m3_pair_rne_sat(y0, y1);
  const uint32_t sign = ((w >> 8) & 0x80u) | ((w >> 16) & 0x8000u);   // bf16 sign bits 15, 31 -> 7, 15
  return m | sign;
}

}  // namespace nvfp4
