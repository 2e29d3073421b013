// The gated activation and its gradient in fp32, for the products whose sums are
// plain fp32 (bf16 and int8 operands).
#pragma once

#include <cuda_runtime.h>

namespace ep {

// s = 1 / (1 + exp(-gate)) and 1 - s, both from t = exp(-|gate|), which neither overflows nor cancels.  The divisor is in
// [1, 2], so an approximate reciprocal and one Newton step give the quotient to an ulp without a division's checks.
// kRounded: for results that are rounded to bf16 at once, without that step and by the short exponential, whose argument's
// own rounding leaves t |gate| 2^-23 off or so (2^-16 where t is 2^-126): a third of the activation's instructions.
template <bool kRounded>
__device__ __forceinline__ void sigmoid_and_rest(float gate, float& s, float& rest) {
    const float t = kRounded ? __expf(-fabsf(gate)) : expf(-fabsf(gate)), d = 1.0f + t;
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(d));
    if (!kRounded) r = fmaf(r, fmaf(-d, r, 1.0f), r);
    const float small = t * r;
    s = gate >= 0.0f ? r : small;
    rest = gate >= 0.0f ? small : r;
}

// gate / (1 + exp(-gate)) * up
template <bool kRounded>
__device__ __forceinline__ float gated_unit(float gate, float up) {
    float s, rest;
    sigmoid_and_rest<kRounded>(gate, s, rest);
    return gate * s * up;
}

// Gradients of the above with respect to gate and up, times gh.
template <bool kRounded>
__device__ __forceinline__ float2 gated_unit_gradient(float gh, float gate, float up) {
    float s, rest;
    sigmoid_and_rest<kRounded>(gate, s, rest);
    return make_float2(gh * up * (s * fmaf(gate, rest, 1.0f)), gh * (gate * s));
}

}  // namespace ep
