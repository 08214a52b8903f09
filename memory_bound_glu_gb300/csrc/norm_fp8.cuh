// norm_fp8.cuh -- residual addition, zero-centred RMSNorm and the e4m3 output
// with a scale per 128 columns, in one pass; and the e4m3 form of a weight.
//
//   s = bf16(x + residual)                        (the residual stream's update)
//   v = s (mean_k s^2 + eps)^-1/2 (1 + w)          fp32, not rounded to bf16
//   scale = max(amax_128(|v|) / 448, 2^-126),  q = e4m3(v / scale)
//
// Memory-bound: 2 + 2 bytes in, 2 + 1 out per element.  A block owns a row and
// keeps it in registers between the statistic and the output, so each byte
// moves once.  The division by the scale is a product with 1 / scale: at most
// 1.5 fp32 ulps before a rounding to 4 bits.
#pragma once

#include "dense_common.cuh"

namespace mbglu {

struct NormFp8Params {
    const uint16_t *x;
    int64_t ldx;
    const uint16_t *residual;
    int64_t ldr;
    uint16_t *residual_out;
    int64_t ldro;
    const uint16_t *w;
    float eps;
    uint8_t *q;
    int64_t ldq;
    float *scale;
    int64_t lds;
    int M, K;
};

// Sum over the block (warps up to 32), the same in every thread; the order of
// the additions is fixed.
__device__ __forceinline__ float block_sum(float v, float *red)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    const int nw = blockDim.x >> 5;
    v = 0.0f;
    for (int i = 0; i < nw; ++i) v += red[i];
    return v;
}

// Any K, stride and 2-byte alignment: the row is read back from residual_out
// for the output (each block reads what it wrote itself).  A thread sums the
// same columns in the same order as in norm_fp8_kernel, so that a row's result
// does not depend on where its operands lie.
__global__ void __launch_bounds__(256) norm_fp8_any_kernel(const NormFp8Params p)
{
    __shared__ float red[8];
    grid_dependency_wait();
    grid_launch_dependents();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, T = static_cast<int>(blockDim.x);
    const int64_t m = blockIdx.x;
    uint16_t *ro = p.residual_out + m * p.ldro;
    float ss = 0.0f;
    for (int64_t k0 = threadIdx.x * 8; k0 < p.K; k0 += T * 8) {
        const int n = static_cast<int>(p.K - k0 < 8 ? p.K - k0 : 8);
        for (int i = 0; i < n; ++i) {
            const uint16_t s = f32_to_bf16(bf16_to_f32(p.x[m * p.ldx + k0 + i]) + bf16_to_f32(p.residual[m * p.ldr + k0 + i]));
            ro[k0 + i] = s;
            const float f = bf16_to_f32(s);
            ss = fmaf(f, f, ss);
        }
    }
    const float inv = rsqrtf(block_sum(ss, red) / static_cast<float>(p.K) + p.eps);   // its barrier: the row is written
    for (int64_t g = warp; g * kScaleBlock < p.K; g += T / 32) {
        float v[4], amax = 0.0f;
#pragma unroll
        for (int b = 0; b < 4; ++b) {
            const int64_t k = g * kScaleBlock + lane + 32 * b;
            v[b] = k < p.K ? bf16_to_f32(ro[k]) * inv * (1.0f + bf16_to_f32(p.w[k])) : 0.0f;
            amax = max_nan(amax, fabsf(v[b]));
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) amax = max_nan(amax, __shfl_xor_sync(0xffffffffu, amax, o));
        const float s = group_scale(amax), r = 1.0f / s;
        if (lane == 0) p.scale[m * p.lds + g] = s;
#pragma unroll
        for (int b = 0; b < 4; ++b) {
            const int64_t k = g * kScaleBlock + lane + 32 * b;
            if (k < p.K) p.q[m * p.ldq + k] = static_cast<uint8_t>(pack_e4m3x2(v[b] * r, 0.0f));
        }
    }
}

// The same for rows of 16-byte chunks (K % 8 == 0, everything 16-byte aligned,
// the output 8): a thread keeps CH chunks of 8 columns in registers between the
// statistic and the output.  Sixteen neighbouring threads hold a group of 128.
template <int CH>
__global__ void __launch_bounds__(256) norm_fp8_kernel(const NormFp8Params p)
{
    __shared__ float red[8];
    const int T = static_cast<int>(blockDim.x), chunks = p.K >> 3;
    grid_dependency_wait();
    grid_launch_dependents();
    const int64_t m = blockIdx.x;
    const uint4 *x = reinterpret_cast<const uint4 *>(p.x + m * p.ldx);
    const uint4 *r = reinterpret_cast<const uint4 *>(p.residual + m * p.ldr);
    const uint4 *w = reinterpret_cast<const uint4 *>(p.w);
    uint4 *ro = reinterpret_cast<uint4 *>(p.residual_out + m * p.ldro);
    uint4 xs[CH], rs[CH], ws[CH];
#pragma unroll
    for (int j = 0; j < CH; ++j) {
        const int c = threadIdx.x + j * T;
        if (c < chunks) {   // residual_out may be x or residual: plain loads
            xs[j] = x[c];
            rs[j] = r[c];
            ws[j] = w[c];
        }
    }
    float v[CH][8], ss = 0.0f;
#pragma unroll
    for (int j = 0; j < CH; ++j) {
        const int c = threadIdx.x + j * T;
        if (c < chunks) {
            const uint32_t xw[4] = {xs[j].x, xs[j].y, xs[j].z, xs[j].w}, rw[4] = {rs[j].x, rs[j].y, rs[j].z, rs[j].w};
            uint32_t o[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                o[i] = pack_bf16x2(bf16_lo(xw[i]) + bf16_lo(rw[i]), bf16_hi(xw[i]) + bf16_hi(rw[i]));
                v[j][2 * i] = bf16_lo(o[i]);
                v[j][2 * i + 1] = bf16_hi(o[i]);
                ss = fmaf(v[j][2 * i], v[j][2 * i], ss);
                ss = fmaf(v[j][2 * i + 1], v[j][2 * i + 1], ss);
            }
            ro[c] = make_uint4(o[0], o[1], o[2], o[3]);
        }
    }
    const float inv = rsqrtf(block_sum(ss, red) / static_cast<float>(p.K) + p.eps);
#pragma unroll
    for (int j = 0; j < CH; ++j) {
        const int c = threadIdx.x + j * T;
        float amax = 0.0f;
        if (c < chunks) {
            const uint32_t ww[4] = {ws[j].x, ws[j].y, ws[j].z, ws[j].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                v[j][2 * i] = v[j][2 * i] * inv * (1.0f + bf16_lo(ww[i]));
                v[j][2 * i + 1] = v[j][2 * i + 1] * inv * (1.0f + bf16_hi(ww[i]));
                amax = max_nan(amax, max_nan(fabsf(v[j][2 * i]), fabsf(v[j][2 * i + 1])));
            }
        }
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) amax = max_nan(amax, __shfl_xor_sync(0xffffffffu, amax, o));
        if (c < chunks) {
            const float s = group_scale(amax), q = 1.0f / s;
            const uint32_t lo = pack_e4m3x4(v[j][0] * q, v[j][1] * q, v[j][2] * q, v[j][3] * q);
            const uint32_t hi = pack_e4m3x4(v[j][4] * q, v[j][5] * q, v[j][6] * q, v[j][7] * q);
            *reinterpret_cast<uint2 *>(p.q + m * p.ldq + 8 * c) = make_uint2(lo, hi);
            if ((c & 15) == 0) p.scale[m * p.lds + (c >> 4)] = s;
        }
    }
}

// A weight [N][K] bf16 to e4m3 with a scale per 128 x 128 block, one thread
// block each: the weight is read twice, two bytes at a time (9728 x 2560: 52 us for
// 75 MB, 1.44 TB/s; the bytes alone would take 11).
// Serving runs it once per weight; training that updates the weights, once per step.
// What it writes may be the very next call's
// weight, which that call's kernel copies before its dependency wait: so it does
// not release its dependents early, and its stores are performed, for
// asynchronous copies too, before a block ends.
__global__ void __launch_bounds__(256) quant_weight_kernel(const uint16_t *w, int64_t ldw, uint8_t *q, int64_t ldq,
                                                           float *scale, int64_t lds, int N, int K)
{
    __shared__ float red[8];
    grid_dependency_wait();
    const int kb = blockIdx.x;
    const int k0 = kb * kScaleBlock;
    for (int64_t nb = blockIdx.y; nb * kScaleBlock < N; nb += gridDim.y) {
        const int64_t n0 = nb * kScaleBlock;
        float amax = 0.0f;
        for (int e = threadIdx.x; e < kScaleBlock * kScaleBlock; e += 256) {
            const int64_t n = n0 + e / kScaleBlock;
            const int k = k0 + e % kScaleBlock;
            if (n < N && k < K) amax = max_nan(amax, fabsf(bf16_to_f32(w[n * ldw + k])));
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) amax = max_nan(amax, __shfl_xor_sync(0xffffffffu, amax, o));
        __syncthreads();   // red of the block before is read
        if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = amax;
        __syncthreads();
        for (int i = 0; i < 8; ++i) amax = max_nan(amax, red[i]);
        const float s = group_scale(amax), r = 1.0f / s;
        if (threadIdx.x == 0) scale[nb * lds + kb] = s;
        for (int e = threadIdx.x; e < kScaleBlock * kScaleBlock; e += 256) {
            const int64_t n = n0 + e / kScaleBlock;
            const int k = k0 + e % kScaleBlock;
            if (n < N && k < K) q[n * ldq + k] = static_cast<uint8_t>(pack_e4m3x2(bf16_to_f32(w[n * ldw + k]) * r, 0.0f));
        }
    }
    __threadfence();
    asm volatile("fence.proxy.async.global;" ::: "memory");
}

}  // namespace mbglu
