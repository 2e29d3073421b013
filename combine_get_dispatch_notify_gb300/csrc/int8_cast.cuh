// int8 casts with one fp32 scale for each row, shared by the casting dispatch and
// the gated product.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

namespace ep {

// Scale of a row whose largest magnitude is `amax` (NaN where the row holds one): amax times fp32's 1 / 127, as torch's
// division by a number does it on a GPU.  The floor keeps the scale of a zero row a normal number, so x / scale is never
// 0 / 0.
__device__ __forceinline__ float row_scale(float amax) {
    constexpr float kFloor = 7.888609052210118e-31f;  // 2^-100
    return (amax == amax ? fmaxf(amax, kFloor) : amax) * (1.0f / 127.0f);
}

// Four quotients in [-127.1, 127.1] -> four int8 bytes, round to nearest even (lowest byte first): 1.5 * 2^23 leaves
// the rounded number in the sum's low bits.
__device__ __forceinline__ uint32_t pack_int8x4(float a, float b, float c, float d) {
    constexpr float kMagic = 12582912.0f;
    const uint32_t lo = __byte_perm(__float_as_uint(__fadd_rn(a, kMagic)), __float_as_uint(__fadd_rn(b, kMagic)), 0x0040);
    const uint32_t hi = __byte_perm(__float_as_uint(__fadd_rn(c, kMagic)), __float_as_uint(__fadd_rn(d, kMagic)), 0x0040);
    return __byte_perm(lo, hi, 0x5410);
}

}  // namespace ep
