// dense_generic.cuh -- the products of the gated block for operands that tensor
// copies cannot take (odd strides or base addresses) and for empty sums: the
// kernel that is right for every case.
//
//   acc0[i, j] = sum_t A0[i, t] B0[t, j]  (+ A1[i, t] B1[t, j])       one accumulator
//   acc0, acc1 = sum_t A0[i, t] B0[t, j],  sum_t A0[i, t] B1[t, j]    DUAL
//
// Every operand has two element strides, so transposed products need no copy.
// bf16 operands, or e4m3 ones that are widened by their block scales when they
// are staged (A: a scale per row and 128 t, B: one per 128 j and 128 t).
// A block of 256 threads owns 16 rows x 128 columns: a warp has two rows, a
// lane columns lane + 32 b, so a row's 128 columns -- one group of an e4m3
// output -- lie in one warp.  fp32 FMAs out of shared memory, one rounding at
// the end.
#pragma once

#include "dense_common.cuh"

namespace mbglu {

enum GenEpilogue { kGenGlu = 0, kGenGrad = 1, kGenPlain = 2, kGenQuant = 3 };

struct GenOperand {
    const void *p;
    int64_t s_out, s_t;      // element strides along the output's index and along t
    const float *scale;      // e4m3: [.., t / 128], row stride lds
    int64_t lds;
};

struct GenParams {
    GenOperand a[2], b[2];
    int rows, cols, T, npair;
    int mode;
    uint16_t *out;           // bf16 outputs (kGenGrad: dG)
    int64_t ldo;
    uint16_t *out2;          // kGenGrad: dU
    float *gu;               // kGenGlu: g and u, [rows][2 cols], or null
    int64_t ldgu;
    const uint16_t *dout;
    int64_t ldd;
    uint8_t *q;
    int64_t ldq;
    float *qs;
    int64_t ldqs;
};

constexpr int kGenRows = 16, kGenCols = 128, kGenT = 32;

template <bool FP8>
__device__ __forceinline__ float gen_fetch(const GenOperand &o, int64_t i, int t, bool block_rows)
{
    const int64_t at = i * o.s_out + t * o.s_t;
    if (!FP8) return bf16_to_f32(static_cast<const uint16_t *>(o.p)[at]);
    const float s = o.scale[(block_rows ? i / kScaleBlock : i) * o.lds + t / kScaleBlock];
    return e4m3_to_f32(static_cast<const uint8_t *>(o.p)[at]) * s;
}

template <int EPI, bool FP8, bool DUAL>
__global__ void __launch_bounds__(256) dense_generic_kernel(const GenParams p)
{
    __shared__ float as[kGenRows][kGenT + 1];
    __shared__ float bs[DUAL ? 2 : 1][kGenT][kGenCols + 1];
    grid_dependency_wait();
    grid_launch_dependents();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int col0 = static_cast<int>(blockIdx.x) * kGenCols;
    const int64_t row_tiles = (static_cast<int64_t>(p.rows) + kGenRows - 1) / kGenRows;
    for (int64_t rt = blockIdx.y; rt < row_tiles; rt += gridDim.y) {
        const int64_t row0 = rt * kGenRows;
        float acc[DUAL ? 2 : 1][2][4] = {};
        for (int pr = 0; pr < (DUAL ? 1 : p.npair); ++pr) {
            for (int t0 = 0; t0 < p.T; t0 += kGenT) {
                __syncthreads();
                for (int e = threadIdx.x; e < kGenRows * kGenT; e += 256) {
                    const int i = e / kGenT, t = e % kGenT;
                    as[i][t] = row0 + i < p.rows && t0 + t < p.T ? gen_fetch<FP8>(p.a[pr], row0 + i, t0 + t, false) : 0.0f;
                }
#pragma unroll
                for (int d = 0; d < (DUAL ? 2 : 1); ++d)
                    for (int e = threadIdx.x; e < kGenCols * kGenT; e += 256) {
                        const int j = e / kGenT, t = e % kGenT;
                        bs[d][t][j] = col0 + j < p.cols && t0 + t < p.T
                                          ? gen_fetch<FP8>(p.b[DUAL ? d : pr], col0 + j, t0 + t, true)
                                          : 0.0f;
                    }
                __syncthreads();
#pragma unroll 8
                for (int t = 0; t < kGenT; ++t) {
                    const float a0 = as[2 * warp][t], a1 = as[2 * warp + 1][t];
#pragma unroll
                    for (int d = 0; d < (DUAL ? 2 : 1); ++d)
#pragma unroll
                        for (int b = 0; b < 4; ++b) {
                            const float w = bs[d][t][lane + 32 * b];
                            acc[d][0][b] = fmaf(a0, w, acc[d][0][b]);
                            acc[d][1][b] = fmaf(a1, w, acc[d][1][b]);
                        }
                }
            }
        }
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const int64_t m = row0 + 2 * warp + r;
            if (m >= p.rows) continue;   // the whole warp
            if constexpr (EPI == kGenQuant) {
                float v[4], amax = 0.0f;
#pragma unroll
                for (int b = 0; b < 4; ++b) {
                    v[b] = col0 + lane + 32 * b < p.cols ? silu_f32(acc[0][r][b]) * acc[DUAL ? 1 : 0][r][b] : 0.0f;
                    amax = max_nan(amax, fabsf(v[b]));
                }
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) amax = max_nan(amax, __shfl_xor_sync(0xffffffffu, amax, o));
                const float s = group_scale(amax), inv = 1.0f / s;
                if (lane == 0) p.qs[m * p.ldqs + blockIdx.x] = s;
#pragma unroll
                for (int b = 0; b < 4; ++b)
                    if (col0 + lane + 32 * b < p.cols)
                        p.q[m * p.ldq + col0 + lane + 32 * b] = static_cast<uint8_t>(pack_e4m3x2(v[b] * inv, 0.0f));
            } else {
#pragma unroll
                for (int b = 0; b < 4; ++b) {
                    const int64_t n = col0 + lane + 32 * b;
                    if (n >= p.cols) continue;
                    const float x = acc[0][r][b], y = acc[DUAL ? 1 : 0][r][b];
                    if constexpr (EPI == kGenGlu) {
                        p.out[m * p.ldo + n] = glu_epilogue(x, y, p.mode);
                        if (p.gu) {
                            p.gu[m * p.ldgu + n] = x;
                            p.gu[m * p.ldgu + p.cols + n] = y;
                        }
                    } else if constexpr (EPI == kGenGrad) {
                        float dg, du;
                        glu_gradients(x, y, bf16_to_f32(p.dout[m * p.ldd + n]), dg, du);
                        p.out[m * p.ldo + n] = f32_to_bf16(dg);
                        p.out2[m * p.ldo + n] = f32_to_bf16(du);
                    } else {
                        p.out[m * p.ldo + n] = f32_to_bf16(x);
                    }
                }
            }
        }
    }
}

inline dim3 gen_grid(int rows, int cols)
{
    const int64_t rt = (static_cast<int64_t>(rows) + kGenRows - 1) / kGenRows;
    return dim3(static_cast<unsigned>((cols + kGenCols - 1) / kGenCols), static_cast<unsigned>(rt < 32768 ? rt : 32768));
}

}  // namespace mbglu
