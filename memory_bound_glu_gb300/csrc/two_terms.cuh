// two_terms.cuh -- fp32 numbers as two bf16 terms, for operands of the tensor cores that one
// term would round too far (an adapter's p, an expert's activation).
#pragma once
#include "glu_math.cuh"

namespace mbglu {

// x and y as two bf16 terms each, hi + lo, off by 2^-18 (each term by half a step of what is left
// to it).  hi stops at the largest bf16 number: what is above it in fp32 is left to lo, and so is
// an infinity, whose second term would else be inf - inf.  NaN is left to lo.
__device__ __forceinline__ void split_bf16x2(float x, float y, uint32_t &hi, uint32_t &lo)
{
    constexpr float kMost = 0x1.fep127f;
    hi = pack_bf16x2(fminf(fmaxf(x, -kMost), kMost), fminf(fmaxf(y, -kMost), kMost));
    lo = pack_bf16x2(x - bf16_lo(hi), y - bf16_hi(hi));
}

}  // namespace mbglu
