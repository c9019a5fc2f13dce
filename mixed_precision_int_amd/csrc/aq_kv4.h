// The 4-bit cache's words: device code shared by the append, the read and the
// attention kernels.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace aq {

// The least word (as a whole number) that holds no scale: 2^64; larger ones are larger
// scales, infinity, NaN and the negative numbers.
constexpr uint32_t kNoScale = 0x5F800000u;
constexpr uint32_t kNaNWord = 0x7FC00000u;
// A word's scale; NaN where it holds none.
__device__ __forceinline__ float scale_held(uint32_t w) { return __uint_as_float(w < kNoScale ? w & ~15u : kNaNWord); }

}  // namespace aq
