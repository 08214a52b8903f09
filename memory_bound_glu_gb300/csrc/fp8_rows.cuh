// fp8_rows.cuh -- the e4m3 products for few rows (a decode step): bound by the
// bytes of the weights, each read once.
//
// mma.sync m16n8k32 with the weights as the 16-row operand and the activations
// as the 8 columns.  Fragments come straight from global memory: within a scale
// block of 128 a lane owns bytes 16 t .. and 64 + 16 t .. (16 each) of a weight
// row -- the order in which the products take the inner index is free, as long
// as both operands use the same -- so a weight fragment is two 16-byte loads per
// row and block, each warp's load takes whole sectors (with 32 consecutive bytes
// per lane every sector was asked for twice), and nothing passes through shared
// memory.  A warp streams one K-slice of 16 rows (of both weights where there
// are two), one or two blocks ahead; slices are joined in shared memory in a
// fixed order.  R groups of 16 rows x S slices = the block's warps.
// An e4m3 output's group of 128 columns is a cluster of 8 / R blocks, which
// exchange their maxima through distributed shared memory.
#pragma once

#include "dense_common.cuh"
#include "tcgen05.cuh"

namespace mbglu {

constexpr int kRowsMax = 16;     // activations' rows

struct Fp8RowsParams {
    const uint8_t *a;
    int64_t lda;
    const float *as;
    int64_t ldas;
    const uint8_t *w[2];
    int64_t ldw[2];
    const float *ws[2];
    int64_t ldws[2];
    int M, N, K;
    int pitch;               // bytes between activation rows in shared memory (rows_pitch)
    int slices;              // S, a power of two up to the warps of a block; R = warps / S
    int prefetch;            // the first weight blocks are requested before the dependency wait
    uint16_t *out;
    int64_t ldo;
    uint8_t *q;
    int64_t ldq;
    float *qs;
    int64_t ldqs;
};

__device__ __forceinline__ uint4 ldg_stream16(const uint8_t *p)
{
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    return v;
}

// Activation rows in shared memory: 64 bytes past a multiple of 128, so that
// the two rows of a quarter-warp's load lie in different halves of the banks.
__host__ __device__ constexpr int rows_pitch(int K) { return (K + 127) / 128 * 128 + 64; }

// All activations, then their scales, then the weights' scales of one block row
// (fp32): what a block keeps in shared memory.
__host__ __device__ constexpr int64_t rows_smem(int M, int K, int mats)
{
    return static_cast<int64_t>(M) * rows_pitch(K) + (static_cast<int64_t>(M) + mats) * ((K + 127) / 128) * 4;
}

__device__ __forceinline__ bool rows_wait(uint64_t *bar) { return mbar_wait_bounded(bar, 0, kWaitLimitNs); }

__device__ __forceinline__ void mma_e4m3(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1)
{
    asm volatile(
        "mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// NT: tiles of 8 activation rows.  OUT: 0 bf16 product, 1 bf16 gated, 2 e4m3
// gated.  WARPS per block, DEPTH scale blocks in flight per warp, and PER_SM
// blocks per SM that the registers must allow.
template <int NT, int OUT, int kRowsWarps, int kRowsDepth, int PER_SM>
__global__ void __launch_bounds__(kRowsWarps * 32, PER_SM) fp8_rows_kernel(const Fp8RowsParams p)
{
    constexpr int MAT = OUT == 0 ? 1 : 2;
    constexpr int MP = 8 * NT;                           // activation rows, padded
    // one slice's sums of one group: [mat][16 rows][MP + 1]
    constexpr int kPart = MAT * 16 * (MP + 1);
    __shared__ float part[kRowsWarps][kPart];
    __shared__ float vals[OUT == 2 ? MP * 128 : 1];      // the gated values, [m][columns of the block]
    __shared__ float peaks[OUT == 2 ? 8 * MP : 1];       // [block of the cluster][m]
    extern __shared__ __align__(128) unsigned char rows_raw[];
    __shared__ uint64_t xbar;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = lane >> 2, t = lane & 3;
    const int S = p.slices, R = kRowsWarps / S;
    const int group = warp / S, slice = warp % S;
    const int kb = (p.K + kScaleBlock - 1) / kScaleBlock;
    const int b0 = kb * slice / S, b1 = kb * (slice + 1) / S;
    const int n0 = (static_cast<int>(blockIdx.x) * R + group) * 16;    // this warp's rows of the weights
    const bool live = n0 < p.N;
    const int r0 = min(n0 + g, p.N - 1), r1 = min(n0 + g + 8, p.N - 1);

    const uint8_t *w0[MAT], *w1[MAT];
#pragma unroll
    for (int d = 0; d < MAT; ++d) {
        w0[d] = p.w[d] + r0 * p.ldw[d] + t * 16;
        w1[d] = p.w[d] + r1 * p.ldw[d] + t * 16;
    }
    uint4 w[kRowsDepth][MAT][4];
    auto load_w = [&](uint4 (&dst)[MAT][4], int b) {
        // K is a multiple of 16: 16 bytes lie in the row or past it, where the
        // activations are 0 and any finite weight will do (the row's start)
        const int k = b * kScaleBlock;
        const int k0 = k + t * 16 < p.K ? k : -t * 16, k1 = k + t * 16 + 64 < p.K ? k + 64 : -t * 16;
#pragma unroll
        for (int d = 0; d < MAT; ++d) {
            dst[d][0] = ldg_stream16(w0[d] + k0);
            dst[d][1] = ldg_stream16(w0[d] + k1);
            dst[d][2] = ldg_stream16(w1[d] + k0);
            dst[d][3] = ldg_stream16(w1[d] + k1);
        }
    };
    unsigned char *xs = rows_raw;
    float *sa = reinterpret_cast<float *>(rows_raw + p.M * p.pitch), *sw = sa + p.M * kb;
    if (threadIdx.x == 0) {
        mbar_init(&xbar, 1);
        fence_mbar_init();
    }
    if (!p.prefetch) grid_dependency_wait();
    if (live) {
#pragma unroll
        for (int i = 0; i < kRowsDepth; ++i)
            if (b0 + i < b1) load_w(w[i], b0 + i);
    }
    // a block's weight rows lie in one row of scale blocks
    const int swrow = min(static_cast<int>(blockIdx.x) * R * 16, p.N - 1) / kScaleBlock;
    for (int i = threadIdx.x; i < MAT * kb; i += kRowsWarps * 32) {
        const int d = i / kb, b = i - d * kb;
        sw[i] = __ldg(p.ws[d] + swrow * p.ldws[d] + b);
    }
    if (p.prefetch) grid_dependency_wait();
    grid_launch_dependents();
    // the activations once per block: the loop would else wait for L2 at every
    // scale block
    if (threadIdx.x == 0) {
        mbar_arrive_expect_tx(&xbar, static_cast<uint32_t>(p.M) * static_cast<uint32_t>(p.K));
        for (int m = 0; m < p.M; ++m) bulk_g2s_plain(xs + m * p.pitch, p.a + m * p.lda, static_cast<uint32_t>(p.K), &xbar);
    }
    for (int i = threadIdx.x; i < p.M * kb; i += kRowsWarps * 32) {
        const int m = i / kb, b = i - m * kb;
        sa[i] = p.as[m * p.ldas + b];
    }
    __syncthreads();
    if (!rows_wait(&xbar)) {
        atomicExch(&g_dense_error, kErrTimeout);
        rows_wait(&xbar);   // no copy may be in flight when the block leaves
    }

    float total[MAT][NT][4] = {};
    if (live) {
#pragma unroll 1
        for (int b = b0; b < b1; b += kRowsDepth) {
#pragma unroll
            for (int i = 0; i < kRowsDepth; ++i) {
                if (b + i >= b1) break;
                const int k = (b + i) * kScaleBlock + t * 16;
                float f[MAT];
#pragma unroll
                for (int d = 0; d < MAT; ++d) f[d] = sw[d * kb + b + i];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    const int m = nt * 8 + g;
                    uint4 x0 = make_uint4(0, 0, 0, 0), x1 = x0;
                    if (m < p.M) {
                        const uint4 *x = reinterpret_cast<const uint4 *>(xs + m * p.pitch + k);
                        if (k < p.K) x0 = x[0];
                        if (k + 64 < p.K) x1 = x[4];
                    }
                    // the scales of the two activation rows of this lane's sums
                    const int m0 = nt * 8 + 2 * t;
                    const float s0 = m0 < p.M ? sa[m0 * kb + b + i] : 0.0f;
                    const float s1 = m0 + 1 < p.M ? sa[(m0 + 1) * kb + b + i] : 0.0f;
#pragma unroll
                    for (int d = 0; d < MAT; ++d) {
                        const uint4 *q = w[i][d];
                        float c[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                        mma_e4m3(c, q[0].x, q[2].x, q[0].y, q[2].y, x0.x, x0.y);
                        mma_e4m3(c, q[0].z, q[2].z, q[0].w, q[2].w, x0.z, x0.w);
                        mma_e4m3(c, q[1].x, q[3].x, q[1].y, q[3].y, x1.x, x1.y);
                        mma_e4m3(c, q[1].z, q[3].z, q[1].w, q[3].w, x1.z, x1.w);
                        float(&s)[4] = total[d][nt];
                        s[0] = fmaf(f[d] * s0, c[0], s[0]);
                        s[1] = fmaf(f[d] * s1, c[1], s[1]);
                        s[2] = fmaf(f[d] * s0, c[2], s[2]);
                        s[3] = fmaf(f[d] * s1, c[3], s[3]);
                    }
                }
                if (b + i + kRowsDepth < b1) load_w(w[i], b + i + kRowsDepth);
            }
        }
    }
#pragma unroll
    for (int d = 0; d < MAT; ++d)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                part[warp][(d * 16 + g + (i >> 1) * 8) * (MP + 1) + nt * 8 + 2 * t + (i & 1)] = total[d][nt][i];
    __syncthreads();

    // join: warp w takes activation rows w, w + 8, ..; lanes take columns
    const int cols = 16 * R, c0 = static_cast<int>(blockIdx.x) * cols;
    auto joined = [&](int d, int c, int m) {
        const float *q = &part[(c >> 4) * S][(d * 16 + (c & 15)) * (MP + 1) + m];
        float v = 0.0f;
        for (int s = 0; s < S; ++s) v += q[s * kPart];
        return v;
    };
    for (int m = warp; m < p.M; m += kRowsWarps) {
        float amax = 0.0f;
        for (int c = lane; c < cols; c += 32) {
            const int n = c0 + c;
            const float x = joined(0, c, m);
            if (OUT == 0) {
                if (n < p.N) p.out[m * p.ldo + n] = f32_to_bf16(x);
            } else {
                const float v = silu_short(x) * joined(MAT - 1, c, m);
                if (OUT == 1) {
                    if (n < p.N) p.out[m * p.ldo + n] = f32_to_bf16(v);
                } else {
                    vals[m * 128 + c] = v;
                    if (n < p.N) amax = max_nan(amax, fabsf(v));
                }
            }
        }
        if (OUT == 2) {
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) amax = max_nan(amax, __shfl_xor_sync(0xffffffffu, amax, o));
            const uint32_t rank = R < 8 ? cluster_ctarank() : 0u;
            if (R < 8) {   // every block of the cluster gets it
                if (lane < 8 / R) st_cluster_f32(map_to_rank(&peaks[rank * MP + m], static_cast<uint32_t>(lane)), amax);
            } else if (lane == 0) {
                peaks[m] = amax;
            }
        }
    }
    if constexpr (OUT == 2) {
        if (R < 8)
            cluster_sync();   // the maxima are there; nobody's memory is touched after it
        else
            __syncthreads();
        const uint32_t rank = R < 8 ? cluster_ctarank() : 0u;
        for (int m = warp; m < p.M; m += kRowsWarps) {
            float amax = 0.0f;
            for (int i = 0; i < 8 / R; ++i) amax = max_nan(amax, peaks[i * MP + m]);
            const float s = group_scale(amax), inv = 1.0f / s;
            if (rank == 0 && lane == 0) p.qs[m * p.ldqs + c0 / kScaleBlock] = s;
            for (int c = lane; c < cols; c += 32)
                if (c0 + c < p.N) p.q[m * p.ldq + c0 + c] = static_cast<uint8_t>(pack_e4m3x2(vals[m * 128 + c] * inv, 0.0f));
        }
    }
}

}  // namespace mbglu
