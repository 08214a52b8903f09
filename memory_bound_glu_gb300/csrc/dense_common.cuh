// dense_common.cuh -- device helpers of the gated block beyond the decode
// batch: the gradients of the GLU, e4m3 conversions and a group's scale, and
// stores of 32 consecutive columns of one row.
#pragma once
#include <cuda_fp16.h>
#include <cstdint>

#include "glu_math.cuh"
#include "ptx.cuh"

namespace mbglu {

// The translation unit's error word: MBGLU_ERR_TIMEOUT after a bounded wait gave up.
static __device__ int g_dense_error;

constexpr int kScaleBlock = 128;                  // columns (and, for weights, rows) per scale
constexpr float kE4m3Max = 448.0f;
constexpr float kScaleMin = 1.17549435e-38f;      // 2^-126: the scale of a group of zeros

// dG = dout u SiLU'(g), dU = dout SiLU(g), in fp32
__device__ __forceinline__ void glu_gradients(float g, float u, float d, float &dg, float &du)
{
    float s, ds;
    silu_and_derivative(g, s, ds);
    dg = d * u * ds;
    du = d * s;
}

// max that keeps a NaN (fmaxf drops it): a group with a NaN gets a NaN scale
__device__ __forceinline__ float max_nan(float a, float b)
{
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// A group's scale, from the largest magnitude in it.
__device__ __forceinline__ float group_scale(float amax) { return max_nan(amax / kE4m3Max, kScaleMin); }

// Two floats to e4m3, round to nearest even, lo in the low byte; magnitudes
// above 448 (a quotient by the scale can pass it by one fp32 rounding) become
// 448, NaN stays NaN.
__device__ __forceinline__ uint32_t pack_e4m3x2(float lo, float hi)
{
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

__device__ __forceinline__ uint32_t pack_e4m3x4(float a, float b, float c, float d)
{
    return pack_e4m3x2(a, b) | (pack_e4m3x2(c, d) << 16);
}

// e4m3 -> fp32 (exact; through fp16, which holds every e4m3 value)
__device__ __forceinline__ float e4m3_to_f32(uint8_t b)
{
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(b)));
    return __half2float(__ushort_as_half(static_cast<uint16_t>(h & 0xffffu)));
}

// 32 bytes at a 32-byte aligned address in one store
__device__ __forceinline__ void st_global_32B(void *p, const uint32_t *w)
{
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                 "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
}

// 32 bf16 values (16 words, two per word) of one row to p[0..31], of which the
// first `valid` exist.  align: 2 when the row is 32-byte aligned, 1 when 16.
// A thread owns a row, so a warp's stores of one word each touch 32 rows: the
// 32-byte form writes whole sectors.
__device__ __forceinline__ void store_bf16_32(uint16_t *p, const uint32_t (&w)[16], int valid, int align)
{
    if (valid >= 32 && align == 2) {
        st_global_32B(p, &w[0]);
        st_global_32B(p + 16, &w[8]);
    } else if (valid >= 32 && align == 1) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            reinterpret_cast<uint4 *>(p)[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
    } else {
#pragma unroll
        for (int i = 0; i < 32; ++i)
            if (i < valid) p[i] = static_cast<uint16_t>(w[i >> 1] >> ((i & 1) * 16));
    }
}

// 32 fp32 values of one row; align as above
__device__ __forceinline__ void store_f32_32(float *p, const float (&v)[32], int valid, int align)
{
    if (valid >= 32 && align == 2) {
#pragma unroll
        for (int i = 0; i < 4; ++i) st_global_32B(p + 8 * i, reinterpret_cast<const uint32_t *>(&v[8 * i]));
    } else if (valid >= 32 && align == 1) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            reinterpret_cast<float4 *>(p)[i] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
    } else {
#pragma unroll
        for (int i = 0; i < 32; ++i)
            if (i < valid) p[i] = v[i];
    }
}

// 32 bf16 values of one row into floats; missing ones (past valid) are 0
__device__ __forceinline__ void load_bf16_32(const uint16_t *p, float (&v)[32], int valid, int align)
{
    if (valid >= 32 && align >= 1) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint4 q = __ldg(reinterpret_cast<const uint4 *>(p) + i);
            const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                v[8 * i + 2 * j] = bf16_to_f32(static_cast<uint16_t>(w[j]));
                v[8 * i + 2 * j + 1] = bf16_to_f32(static_cast<uint16_t>(w[j] >> 16));
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] = i < valid ? bf16_to_f32(__ldg(p + i)) : 0.0f;
    }
}

}  // namespace mbglu
