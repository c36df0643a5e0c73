// fp8_scale.cuh -- power-of-two scales, for the block quantiser and the 8-bit cache.
#pragma once

#include <cstdint>

namespace gb300 {

// The smallest power of two >= s (s >= 0 finite), normal or subnormal; 0 for 0.
__device__ __forceinline__ float pow2_at_least(float s)
{
    const uint32_t b = __float_as_uint(s);
    if ((b & 0x7F800000u) == 0) {  // subnormal: 2^k >= m * 2^-149 from m's highest bit
        const uint32_t m = b & 0x7FFFFFu;
        return __uint_as_float((m & (m - 1)) == 0 ? m : (1u << (32 - __clz(m))));
    }
    return (b & 0x7FFFFFu) == 0 ? s : __uint_as_float((b & 0x7F800000u) + 0x00800000u);
}

}  // namespace gb300
