// lora_generic.cuh -- products with low-rank adapters for operands that tensor copies
// cannot take: the kernels that are right for every case.
//
//   p[m, j]   = scale[a] sum_k x[m, k] A[a][j, k]              a = adapter[m], j < R
//   acc[m, n] = sum_k x[m, k] W[n, k] + sum_j p[m, j] B[a][n, j]
//
// A row whose index is not in [0, adapters) has no second term; B of other rows'
// adapters never enters a row's sum.  fp32 sums, one rounding at the end.
#pragma once
#include "dense_generic.cuh"

namespace mbglu {

struct LoraSide {
    const uint16_t *w, *a, *b;
    int64_t ldw, a_adapter, lda, b_adapter, ldb;
};

struct LoraParams {
    const uint16_t *x;
    int64_t ldx;
    LoraSide side[2];
    const int32_t *adapter;
    const float *scale;      // null: 1
    float *p;                // [M][sides R]: the second side's from column R on
    uint16_t *terms;         // [2][M][sides R]: p's two bf16 terms
    int32_t *blocks;         // of 32 rows each: their adapter, or that they have none or several; or null
    uint16_t *out;
    int64_t ldo;
    int M, N, K, adapters, R, mode;
};

// the row's adapter, or -1
__device__ __forceinline__ int lora_adapter(const LoraParams &p, int64_t m)
{
    const int a = p.adapters > 0 && m < p.M ? p.adapter[m] : -1;
    return a >= 0 && a < p.adapters ? a : -1;
}

// A warp per p[m, j]; rows without an adapter are left as they are.
template <int SIDES>
__global__ void __launch_bounds__(256) lora_generic_shrink(const LoraParams p)
{
    grid_dependency_wait();
    grid_launch_dependents();
    const int lane = threadIdx.x & 31, cols = SIDES * p.R;
    const int64_t total = static_cast<int64_t>(p.M) * cols;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5); i < total; i += static_cast<int64_t>(gridDim.x) * 8) {
        const int64_t m = i / cols;
        const int j = static_cast<int>(i % cols), a = lora_adapter(p, m);
        if (a < 0) continue;   // the whole warp
        const LoraSide &s = p.side[SIDES == 2 && j >= p.R];
        const uint16_t *x = p.x + m * p.ldx, *w = s.a + a * s.a_adapter + (j >= p.R ? j - p.R : j) * s.lda;
        float v = 0.0f;
        for (int k = lane; k < p.K; k += 32) v = fmaf(bf16_to_f32(x[k]), bf16_to_f32(w[k]), v);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        if (lane == 0) p.p[i] = p.scale ? v * p.scale[a] : v;
    }
}

// dense_generic_kernel's tiles, then the adapter's term of each output.
template <int SIDES>
__global__ void __launch_bounds__(256) lora_generic_kernel(const LoraParams p)
{
    __shared__ float as[kGenRows][kGenT + 1];
    __shared__ float bs[SIDES][kGenT][kGenCols + 1];
    grid_dependency_wait();
    grid_launch_dependents();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t col0 = static_cast<int64_t>(blockIdx.x) * kGenCols;
    const int64_t row_tiles = (static_cast<int64_t>(p.M) + kGenRows - 1) / kGenRows;
    for (int64_t rt = blockIdx.y; rt < row_tiles; rt += gridDim.y) {
        const int64_t row0 = rt * kGenRows;
        float acc[SIDES][2][4] = {};
        for (int t0 = 0; t0 < p.K; t0 += kGenT) {
            __syncthreads();
            for (int e = threadIdx.x; e < kGenRows * kGenT; e += 256) {
                const int i = e / kGenT, t = e % kGenT;
                as[i][t] = row0 + i < p.M && t0 + t < p.K ? bf16_to_f32(p.x[(row0 + i) * p.ldx + t0 + t]) : 0.0f;
            }
#pragma unroll
            for (int d = 0; d < SIDES; ++d)
                for (int e = threadIdx.x; e < kGenCols * kGenT; e += 256) {
                    const int j = e / kGenT, t = e % kGenT;
                    bs[d][t][j] = col0 + j < p.N && t0 + t < p.K ? bf16_to_f32(p.side[d].w[(col0 + j) * p.side[d].ldw + t0 + t]) : 0.0f;
                }
            __syncthreads();
#pragma unroll 8
            for (int t = 0; t < kGenT; ++t) {
                const float a0 = as[2 * warp][t], a1 = as[2 * warp + 1][t];
#pragma unroll
                for (int d = 0; d < SIDES; ++d)
#pragma unroll
                    for (int b = 0; b < 4; ++b) {
                        const float w = bs[d][t][lane + 32 * b];
                        acc[d][0][b] = fmaf(a0, w, acc[d][0][b]);
                        acc[d][1][b] = fmaf(a1, w, acc[d][1][b]);
                    }
            }
        }
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const int64_t m = row0 + 2 * warp + r;
            if (m >= p.M) continue;   // the whole warp
            const int a = lora_adapter(p, m);
#pragma unroll
            for (int b = 0; b < 4; ++b) {
                const int64_t n = col0 + lane + 32 * b;
                if (n >= p.N) continue;
                if (a >= 0) {
#pragma unroll
                    for (int d = 0; d < SIDES; ++d) {
                        const uint16_t *w = p.side[d].b + a * p.side[d].b_adapter + n * p.side[d].ldb;
                        const float *q = p.p + m * SIDES * p.R + d * p.R;
                        float v = 0.0f;
                        for (int j = 0; j < p.R; ++j) v = fmaf(q[j], bf16_to_f32(w[j]), v);
                        acc[d][r][b] += v;
                    }
                }
                if constexpr (SIDES == 2)
                    p.out[m * p.ldo + n] = glu_epilogue(acc[0][r][b], acc[1][r][b], p.mode);
                else
                    p.out[m * p.ldo + n] = f32_to_bf16(acc[0][r][b]);
            }
        }
    }
}

}  // namespace mbglu
