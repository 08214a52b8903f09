// glu_math.cuh -- scalar helpers that every kernel of the library shares: bf16
// conversions, SiLU and its derivative, the GLU epilogue's two rounding modes,
// and the limit of a bounded wait.
#pragma once
#include <cuda_bf16.h>
#include <cstdint>

namespace mbglu {

constexpr uint64_t kWaitLimitNs = 2000000000ull;  // 2 s per bounded wait
constexpr int kErrTimeout = 8;                    // == MBGLU_ERR_TIMEOUT

// ---------------------------------------------------------------------------
// scalar helpers
// ---------------------------------------------------------------------------

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
__device__ __forceinline__ float bf16_to_f32(uint16_t b) { return __uint_as_float(static_cast<uint32_t>(b) << 16); }
__device__ __forceinline__ uint16_t f32_to_bf16(float x) { return __bfloat16_as_ushort(__float2bfloat16_rn(x)); }
__device__ __forceinline__ float round_to_bf16(float x) { return __bfloat162float(__float2bfloat16_rn(x)); }
// two floats rounded to nearest-even bf16 in one paired conversion
// (cvt.rn.bf16x2.f32), lo in the low half
__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi)
{
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&v);
}

// SiLU(x) = x / (1 + e^-x) = x * e^x / (1 + e^x), evaluated with t = e^-|x| so
// that nothing overflows: for x < -88.7 the first form's e^-x is +inf in fp32
// and would flush SiLU to -0, although x * e^x is still a normal bf16 value
// down to x ~ -92 (bf16 keeps fp32's exponent range).  Precise expf and IEEE
// division (no fast math).
__device__ __forceinline__ float silu_f32(float x)
{
    const float t = expf(-fabsf(x));
    return (x >= 0.0f ? x : x * t) / (1.0f + t);
}

// mode 0 (FUSED): one rounding.  mode 1 (HF): the bf16 composite's roundings:
// g, u, SiLU(g) and the product each round to bf16 (PR #9057, section
// "Changes").  sb * ub is exact in fp32.
__device__ __forceinline__ uint16_t glu_epilogue(float g, float u, int mode)
{
    if (mode == 0) return f32_to_bf16(silu_f32(g) * u);
    const float gb = round_to_bf16(g);
    const float ub = round_to_bf16(u);
    const float sb = round_to_bf16(silu_f32(gb));
    return f32_to_bf16(sb * ub);
}

// SiLU(x) and SiLU'(x) = sigma(x) * (1 + x * (1 - sigma(x))), from t = e^-|x|
// so that nothing overflows: sigma = 1/(1+t), 1 - sigma = t/(1+t) for x >= 0,
// and the two swapped below.  Precise expf and IEEE division.
__device__ __forceinline__ void silu_and_derivative(float x, float &silu, float &dsilu)
{
    const float t = expf(-fabsf(x));
    const float sig = (x >= 0.0f ? 1.0f : t) / (1.0f + t);
    const float rest = (x >= 0.0f ? t : 1.0f) / (1.0f + t);   // 1 - sigma
    silu = x * sig;
    dsilu = sig * (1.0f + x * rest);
}

}  // namespace mbglu
