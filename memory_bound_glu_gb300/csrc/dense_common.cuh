// dense_common.cuh -- device helpers of the gated block beyond the decode
// batch.  Its kernels may start before the one ahead of them has ended and then
// wait for it, so what that one may have written is read with plain loads, never
// with read-only ones, whose data may not change while a kernel runs.  Here: the
// gradients of the GLU, e4m3 conversions and a group's scale, and stores of 32
// consecutive columns of one row.
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

// e^-|x|.  With z = |x| log2(e) rounded and r what the rounding left out,
// e^-|x| = 2^-z (1 - r ln 2): relative error below 2^-21 (2^-z alone is off by
// |x| 2^-24) up to |x| = 87.  Beyond, the result is an fp32 subnormal of at most three
// roundings of 2^-149 (at |x| = 100 up to a tenth of it), as expf's would be of one.
// |x| is capped where the result is 0 anyway, so that infinities leave no inf - inf.
__device__ __forceinline__ float exp_neg_abs(float x)
{
    constexpr float kLog2e = 1.44269504f, kLog2eLow = 1.92596299e-8f, kLn2 = 0.693147181f;
    const float a = fminf(fabsf(x), 200.0f);
    const float z = a * kLog2e;
    const float r = fmaf(a, kLog2eLow, fmaf(a, kLog2e, -z));
    float t;
    asm("ex2.approx.f32 %0, %1;" : "=f"(t) : "f"(-z));
    return fmaf(t * r, -kLn2, t);
}

// SiLU(x) in a third of the instructions of the precise form (silu_f32): relative
// error below 2^-20, and for x < -87 an error below |x| 2^-146, which is a bf16 step's
// 2^-133 and more only beside results that bf16 no longer holds.  An epilogue that is unrolled over a thread's 64
// outputs is bound by fetching its instructions once per tile: glu_fp8's at
// M = 48, K = 128 took 17.0 us with the precise form.
__device__ __forceinline__ float silu_short(float x)
{
    const float t = exp_neg_abs(x);
    return __fdividef(x >= 0.0f ? x : x * t, 1.0f + t);
}

// the GLU epilogue's roundings (glu_epilogue) on silu_short
__device__ __forceinline__ uint32_t glu_hf_short(float g, float u)
{
    return f32_to_bf16(round_to_bf16(silu_short(round_to_bf16(g))) * round_to_bf16(u));
}

// dG = dout u SiLU'(g), dU = dout SiLU(g), in fp32: with s the sigmoid,
// SiLU' = s (1 + g (1 - s)).
//
// The callers round both once to bf16, because they are the tensor cores' operands in
// the gradients' products: each gradient then carries two roundings, an error of
// 2.35e-3 in the 2-norm where one rounding leaves 1.66e-3 (333 x 1000 x 2504).  Kept
// whole, as three bf16 terms each (glu_backward, up to 64 rows, where the weights'
// bytes bound it), they would triple products that are bound by the tensor cores.
__device__ __forceinline__ void glu_gradients(float g, float u, float d, float &dg, float &du)
{
    const float t = exp_neg_abs(g), inv = __fdividef(1.0f, 1.0f + t);
    const float s = (g >= 0.0f ? 1.0f : t) * inv, rest = (g >= 0.0f ? t : 1.0f) * inv;
    dg = d * u * (s * fmaf(g, rest, 1.0f));
    du = d * (g * s);
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

// ---- a warp's 32 rows x 32 columns, a thread per row ------------------------------
//
// Rows that lie on 16 bytes move by their own threads: a store of one word each
// touches 32 rows, the 32-byte form writes whole sectors.  Others -- an odd row
// length, the last columns -- go through `buf` (shared memory, kRowBuf words per
// warp), a row at a time with consecutive columns in consecutive lanes: 32 two-byte
// stores to 32 rows each took 869 x 12359 outputs 123 us, this way 29.
//
// p: the warp's first row, first column; rows: how many of the 32 exist (may be 0
// or less); valid: columns (1 or more); align: 2 where every row lies on 32 bytes, 1
// on 16.  The whole warp calls.
constexpr int kRowBuf = 32 * 17;

__device__ __forceinline__ void warp_store_bf16(uint32_t *buf, uint16_t *p, int64_t ld, const uint32_t (&w)[16], int rows,
                                                int valid, int align)
{
    const int lane = threadIdx.x & 31;
    if (align > 0 && valid >= 32) {
        if (lane >= rows) return;
        uint16_t *q = p + lane * ld;
        if (align == 2) {
            st_global_32B(q, &w[0]);
            st_global_32B(q + 16, &w[8]);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                reinterpret_cast<uint4 *>(q)[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) buf[lane * 17 + i] = w[i];
    __syncwarp();
    const int n = min(rows, 32);
#pragma unroll 4
    for (int r = 0; r < n; ++r)
        if (lane < valid) p[r * ld + lane] = static_cast<uint16_t>(buf[r * 17 + (lane >> 1)] >> ((lane & 1) * 16));
    __syncwarp();
}

__device__ __forceinline__ void warp_store_f32(uint32_t *buf, float *p, int64_t ld, const uint32_t (&v)[32], int rows, int valid,
                                               int align)
{
    const int lane = threadIdx.x & 31;
    if (align > 0 && valid >= 32) {
        if (lane >= rows) return;
        float *q = p + lane * ld;
        if (align == 2) {
#pragma unroll
            for (int i = 0; i < 4; ++i) st_global_32B(q + 8 * i, &v[8 * i]);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                reinterpret_cast<uint4 *>(q)[i] = make_uint4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
        }
        return;
    }
    const int n = min(rows, 32);
#pragma unroll
    for (int h = 0; h < 2; ++h) {   // 16 columns at a time, two rows per store
#pragma unroll
        for (int i = 0; i < 16; ++i) buf[lane * 17 + i] = v[16 * h + i];
        __syncwarp();
        const int c = lane & 15;
#pragma unroll 4
        for (int r = lane >> 4; r < n; r += 2)
            if (16 * h + c < valid) p[r * ld + 16 * h + c] = __uint_as_float(buf[r * 17 + c]);
        __syncwarp();
    }
}

__device__ __forceinline__ void warp_store_e4m3(uint32_t *buf, uint8_t *p, int64_t ld, const uint32_t (&w)[8], int rows, int valid,
                                                int align)
{
    const int lane = threadIdx.x & 31;
    if (align > 0 && valid >= 32) {
        if (lane >= rows) return;
        uint8_t *q = p + lane * ld;
        if (align == 2) {
            st_global_32B(q, w);
        } else {
            reinterpret_cast<uint4 *>(q)[0] = make_uint4(w[0], w[1], w[2], w[3]);
            reinterpret_cast<uint4 *>(q)[1] = make_uint4(w[4], w[5], w[6], w[7]);
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) buf[lane * 9 + i] = w[i];
    __syncwarp();
    const int n = min(rows, 32);
#pragma unroll 4
    for (int r = 0; r < n; ++r)
        if (lane < valid) p[r * ld + lane] = static_cast<uint8_t>(buf[r * 9 + (lane >> 2)] >> ((lane & 3) * 8));
    __syncwarp();
}

// This thread's row as floats; what does not exist is 0.
__device__ __forceinline__ void warp_load_bf16(uint32_t *buf, const uint16_t *p, int64_t ld, float (&v)[32], int rows, int valid,
                                               int align)
{
    const int lane = threadIdx.x & 31;
    uint32_t w[16];
    if (align > 0 && valid >= 32) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint4 q = lane < rows ? reinterpret_cast<const uint4 *>(p + lane * ld)[i] : make_uint4(0, 0, 0, 0);
            w[4 * i] = q.x;
            w[4 * i + 1] = q.y;
            w[4 * i + 2] = q.z;
            w[4 * i + 3] = q.w;
        }
    } else {
        uint16_t *half = reinterpret_cast<uint16_t *>(buf);   // rows of 34
#pragma unroll 4
        for (int r = 0; r < 32; ++r) half[r * 34 + lane] = r < rows && lane < valid ? p[r * ld + lane] : static_cast<uint16_t>(0);
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 16; ++i) w[i] = buf[lane * 17 + i];
        __syncwarp();
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        v[2 * i] = bf16_lo(w[i]);
        v[2 * i + 1] = bf16_hi(w[i]);
    }
}

}  // namespace mbglu
