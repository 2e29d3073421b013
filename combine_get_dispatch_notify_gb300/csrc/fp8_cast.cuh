// e4m3 casts with one fp32 scale per block of 128 columns, shared by the
// casting dispatch and the gated product.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

namespace ep {

constexpr int kScaleBlock = 128;  // columns that share one scale

__host__ __device__ constexpr int scale_blocks(int n) { return (n + kScaleBlock - 1) / kScaleBlock; }

// Scale of a block whose largest magnitude is `amax`.  The floor keeps the
// scale of a zero (or vanishing) block a normal number, so x / scale is never
// 0 / 0.  A block whose largest magnitude is below 2^-100 (bf16 and fp32 go down
// to 2^-133 and 2^-149) gets the same scale and fewer of e4m3's digits, or 0.
__device__ __forceinline__ float block_scale(float amax) {
    constexpr float kFloor = 7.888609052210118e-31f;  // 2^-100
    return fmaxf(amax, kFloor) / 448.0f;
}

// x / scale as the division rounds it, by the reciprocal `inv` = 1 / scale, itself rounded by a division: the product is
// corrected by its exact remainder, which brings it within one ulp, and from there a second time, which gives the nearest
// number (Markstein).  An infinite scale leaves 0, or NaN of an infinity, as the division does.  Below scales of about
// 2^-90 the remainders lose bits, and a quotient beside a tie may round to its other side.
__device__ __forceinline__ float over_scale(float x, float scale, float inv) {
    const float q = x * inv;
    float c = fmaf(fmaf(-q, scale, x), inv, q);
    c = fmaf(fmaf(-c, scale, x), inv, c);
    return c == c ? c : q;
}

// Four floats -> four e4m3 bytes, round to nearest even (lowest byte first).
__device__ __forceinline__ uint32_t pack_e4m3x4(float a, float b, float c, float d) {
    uint16_t lo, hi;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
    return static_cast<uint32_t>(lo) | (static_cast<uint32_t>(hi) << 16);
}

}  // namespace ep
