// The activation that an int8 code stands for: bf16(q / x_scale), one correctly
// rounded fp32 division (row_div.hpp's multiply and two fused steps).  A scale
// under that form's range (rows beyond 2^107) is first brought into it by an
// exact factor of 2^64, which the quotient gets back: exact too, or the same
// overflow.  Scales are taken to be at most 2^100 (the codes' are at most
// 127 / 1e-5).
#pragma once

#include "common.hpp"

namespace bl {

struct RestoreRow {
  float d, y, post;
};

__device__ __forceinline__ RestoreRow restore_row(float x_scale) {
  RestoreRow r;
  const bool small = x_scale < 7.888609052210118e-31f;  // 2^-100
  r.d = small ? x_scale * 18446744073709551616.0f : x_scale;
  r.post = small ? 18446744073709551616.0f : 1.0f;
  r.y = 1.0f / r.d;
  return r;
}

// Codes in bytes `lo` and `lo + 1` of w, restored, as a dword of two bf16.
__device__ __forceinline__ uint32_t restore2(uint32_t w, int lo, const RestoreRow& r) {
  const float a = (float)(int8_t)(w >> (8 * lo)), b = (float)(int8_t)(w >> (8 * lo + 8));
  return pack_bf16x2(row_div_fast(a, r.d, r.y) * r.post, row_div_fast(b, r.d, r.y) * r.post);
}

}  // namespace bl
