// Largest magnitudes of weights, for their scales (w4.hip, w8.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace bl {

// |x| as bits: whole numbers in the order of the magnitudes, infinity above them and
// NaN above that, so that a maximum of them keeps a NaN (fmaxf drops it).
__device__ __forceinline__ uint32_t magnitude_bits(float x) { return __float_as_uint(x) & 0x7FFFFFFFu; }

}  // namespace bl
