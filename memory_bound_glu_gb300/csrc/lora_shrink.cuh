// lora_shrink.cuh -- the first half of the adapters' term: p[m, j] = scale[a] sum_k x[m, k]
// A[a][j, k] with a = adapter[m], on the tensor cores of single warps (mma.sync).
//
// A block takes 16 MT rows and 8 NT of the rank's columns; the warps of its cluster split
// the inner dimension and add up in shared memory, in order.  For each adapter that occurs
// among the rows it runs the product of all of them with that adapter's A and writes the
// rows that use it: a product of an adapter's 8 columns with one row costs as much as with
// sixteen, and rows of a decode batch mostly have an adapter of their own (few rows: a
// cluster per adapter, so that they run side by side).  Which k sits in which place of a
// fragment is free as long as both operands agree, so a lane reads 16 consecutive bytes of
// a row, enough for two steps of 16.
//
// p is written in fp32, and as two bf16 terms (off by 2^-18) for the tensor cores.  Beside
// it a table with a number for 32 rows each: their adapter where all of them have the same,
// kNoAdapter, or kMixed.
#pragma once
#include "lora_generic.cuh"
#include "stack_copy.cuh"
#include "tcgen05.cuh"
#include "two_terms.cuh"

namespace mbglu {

__device__ __forceinline__ void mma_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

constexpr int kShrinkWarps = 8;
constexpr int kLoraBlock = 32;                    // rows per entry of the table
constexpr int kNoAdapter = -1, kMixed = -2;

// the warps' sums, then the block's
template <int MT, int NT>
constexpr uint32_t shrink_smem()
{
    return (kShrinkWarps + 1) * MT * 16 * (NT * 8 + 4) * 4;
}

__device__ __forceinline__ float ld_cluster_f32(uint32_t addr)
{
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}

// blockIdx: (column tiles of all sides x the cluster's blocks, row groups, adapters side by side)
template <int SIDES, int MT, int NT, int UNROLL>
__global__ void __launch_bounds__(kShrinkWarps * 32) lora_shrink_kernel(const LoraParams p, const int split)
{
    extern __shared__ float shrink_part[];
    constexpr int kRows = MT * 16, kCols = NT * 8, kPitch = kCols + 4;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, row = lane >> 2, quad = lane & 3;
    const int rank = split > 1 ? static_cast<int>(blockIdx.x) % split : 0, col = static_cast<int>(blockIdx.x) / split;
    const int tiles = (p.R + kCols - 1) / kCols, which = SIDES == 2 && col >= tiles ? 1 : 0;
    const LoraSide &side = p.side[which];
    const int j0 = (col - which * tiles) * kCols, width = SIDES * p.R;
    const int steps = (p.K + 31) / 32, warps = kShrinkWarps * split, w0 = rank * kShrinkWarps + warp;
    const int s0 = steps * w0 / warps, s1 = steps * (w0 + 1) / warps;
    float *total = shrink_part + kShrinkWarps * kRows * kPitch;
    grid_dependency_wait();
    grid_launch_dependents();   // behind the wait: lora_pair_kernel reads x then (LoraPairParams::early)
    for (int64_t group = blockIdx.y; group * kRows < p.M; group += gridDim.y) {
        const int64_t m0 = group * kRows;
        const int mine = lane < kRows ? lora_adapter(p, m0 + lane) : -1;   // kRows <= 32
        uint32_t left = __ballot_sync(0xffffffffu, mine >= 0);
        if (p.blocks && m0 % kLoraBlock == 0 && blockIdx.x == 0 && blockIdx.z == 0 && warp == 0) {
            // rows behind the last agree with any
            const uint32_t in = __ballot_sync(0xffffffffu, m0 + lane < p.M);
            const int its = lora_adapter(p, m0 + lane), a = __shfl_sync(0xffffffffu, its, 0);
            const uint32_t same = __ballot_sync(0xffffffffu, its == a);
            if (lane == 0) p.blocks[m0 / kLoraBlock] = (in & ~same) ? kMixed : a;
        }
        for (uint32_t nth = 0; left; ++nth) {
            const int a = __shfl_sync(0xffffffffu, mine, __ffs(left) - 1);
            const uint32_t rows = __ballot_sync(0xffffffffu, mine == a);
            left &= ~rows;
            if (nth % gridDim.z != blockIdx.z) continue;
            const float scale = p.scale ? p.scale[a] : 1.0f;
            float acc[MT][NT][4] = {};
            const uint16_t *w = side.a + a * side.a_adapter + (j0 + row) * side.lda;
            const uint16_t *x = p.x + (m0 + row) * p.ldx;
#pragma unroll UNROLL
            for (int s = s0; s < s1; ++s) {
                const int k = s * 32 + quad * 8;
                uint4 xa[MT][2], wb[NT];
#pragma unroll
                for (int i = 0; i < MT; ++i)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const int r = i * 16 + h * 8;
                        // only rows that use the adapter are read
                        xa[i][h] = k < p.K && (rows >> (r + row) & 1u) ? *reinterpret_cast<const uint4 *>(x + r * p.ldx + k) : make_uint4(0, 0, 0, 0);
                    }
#pragma unroll
                for (int n = 0; n < NT; ++n)
                    wb[n] = k < p.K && j0 + n * 8 < p.R ? *reinterpret_cast<const uint4 *>(w + n * 8 * side.lda + k) : make_uint4(0, 0, 0, 0);
#pragma unroll
                for (int i = 0; i < MT; ++i) {
                    const uint32_t a0[4] = {xa[i][0].x, xa[i][1].x, xa[i][0].y, xa[i][1].y};
                    const uint32_t a1[4] = {xa[i][0].z, xa[i][1].z, xa[i][0].w, xa[i][1].w};
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        mma_16816(acc[i][n], a0, wb[n].x, wb[n].y);
                        mma_16816(acc[i][n], a1, wb[n].z, wb[n].w);
                    }
                }
            }
            // the block's warps, then the cluster's blocks.  What is written here was read
            // for the last adapter before the barriers below.
            float *part = shrink_part + warp * kRows * kPitch;
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    float *q = part + (i * 16 + row) * kPitch + n * 8 + quad * 2;
                    q[0] = acc[i][n][0];
                    q[1] = acc[i][n][1];
                    q[8 * kPitch] = acc[i][n][2];
                    q[8 * kPitch + 1] = acc[i][n][3];
                }
            __syncthreads();
            const auto put = [&](int r, int j, float v) {
                v *= scale;
                const int64_t at = (m0 + r) * width + which * p.R + j0 + j;
                p.p[at] = v;
                uint32_t hi, lo;
                split_bf16x2(v, 0.0f, hi, lo);
                p.terms[at] = static_cast<uint16_t>(hi);
                p.terms[at + p.M * static_cast<int64_t>(width)] = static_cast<uint16_t>(lo);
            };
            for (int e = threadIdx.x; e < kRows * kCols; e += kShrinkWarps * 32) {
                const int r = e / kCols, j = e % kCols;
                if (!(rows >> r & 1u) || j0 + j >= p.R) continue;
                float v = 0.0f;
#pragma unroll
                for (int i = 0; i < kShrinkWarps; ++i) v += shrink_part[(i * kRows + r) * kPitch + j];
                if (split == 1)
                    put(r, j, v);
                else
                    total[r * kPitch + j] = v;
            }
            if (split == 1) {
                __syncthreads();
                continue;
            }
            __syncwarp();
            cluster_sync();
            for (int e = threadIdx.x * split + rank; e < kRows * kCols; e += kShrinkWarps * 32 * split) {
                const int r = e / kCols, j = e % kCols;
                if (!(rows >> r & 1u) || j0 + j >= p.R) continue;
                float v = 0.0f;
                for (int i = 0; i < split; ++i) v += ld_cluster_f32(map_to_rank(total + r * kPitch + j, static_cast<uint32_t>(i)));
                put(r, j, v);
            }
            __syncwarp();
            cluster_sync();
        }
    }
}

}  // namespace mbglu
