// fp8_pair.cuh -- the products of e4m3 operands with block scales on CTA pairs:
// the pipeline of pair_gemm.cuh with 128 bytes of the inner dimension per
// stage, so that a stage is one scale block.
//
//   out[m, n] = sum_b sa[m, b] sw[n / 128, b] sum_{k in block b} a[m, k] w[n, k]
//
// The inner sum of a block is formed by the tensor cores in one of two
// tensor-memory buffers; while the next block runs into the other, the eight
// epilogue warps read it (128 columns per thread and block), scale it and add
// it to fp32 totals in registers.  A thread's columns lie in one 128-row block
// of the weight (or 64 + 64 in one block of each weight), so the scale of a
// block is one or two products per thread.
//
// What bounds it: the reading and scaling.  4096 x 4864 x 11008 takes 157 us
// (2.79 PFLOP/s, 460 ns per block and tile); with half of the FMAs left out it
// took 147, with one in sixteen 131, with the blocks summed in tensor memory and
// no scaling at all about 110 (timed copies).  The MMAs alone would take 270 ns
// per block and tile at the dense e4m3 rate.
#pragma once

#include "pair_gemm.cuh"

namespace mbglu {

enum Fp8Epilogue { kFp8Out = 0, kFp8Glu = 1, kFp8GluQuant = 2 };

struct Fp8PairParams {
    PairPlan plan;
    const float *as;          // a's scales
    int64_t ldas;
    const float *ws[2];       // the weights' scales
    int64_t ldws[2];
    int wblocks;              // scale rows of a weight
    uint16_t *out;
    int64_t ldo;
    int out_align;
    uint8_t *q;
    int64_t ldq;
    int q_align;
    float *qs;
    int64_t ldqs;
    float *part;
};

// The scales of 8 blocks at a time, staged by an otherwise idle warp: a thread's
// own row of a's scales is one line per lane and load, which costs the epilogue
// 32 cache accesses per warp and block (4096 x 4864 x 11008: 238 us against
// 195 us from shared memory).
constexpr int kScaleGroup = 8;
struct ScaleStage {
    float a[kScaleGroup][132];   // this CTA's rows; 4 words of padding spread a load over the banks
    float w[2][kScaleGroup];     // weights: blocks 2 ni and 2 ni + 1, or gate and up
};
constexpr uint32_t kFp8Smem = kPairSmem + 2 * sizeof(ScaleStage);

// Two fp32 in one 64-bit register, as the packed FMA takes them.
__device__ __forceinline__ uint64_t pack_f32x2(float lo, float hi)
{
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ float2 unpack_f32x2(uint64_t v)
{
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}

// acc += f (lo, hi), one packed FMA.  Volatile: kept in order with the loads
// around it, so that no more than two steps' columns are held at a time.
__device__ __forceinline__ void scale_add(uint64_t &acc, uint32_t lo, uint32_t hi, uint64_t f)
{
    asm volatile(
        "{\n\t.reg .b64 a;\n\t"
        "mov.b64 a, {%1, %2};\n\t"
        "fma.rn.f32x2 %0, a, %3, %0;\n\t}"
        : "+l"(acc)
        : "r"(lo), "r"(hi), "l"(f));
}

template <int EPI>
__global__ void __launch_bounds__(kPairThreads, 1) fp8_pair_kernel(const Fp8PairParams p, const __grid_constant__ PairMaps maps)
{
    constexpr bool kDual = EPI != kFp8Out;
    constexpr int kMode = kDual ? kPairDual : kPairSum;
    extern __shared__ unsigned char pair_raw[];
    const PairShared s = pair_shared(pair_raw);
    const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();
    ScaleStage *scales = reinterpret_cast<ScaleStage *>(s.row_bufs + kPairRowBufs / 4);
    uint64_t *scale_full = reinterpret_cast<uint64_t *>(s.slot + 2), *scale_empty = scale_full + 2;
    if (threadIdx.x == 32) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(&scale_full[i], 1);
            mbar_init(&scale_empty[i], 8);
        }
        fence_mbar_init();
    }
    const uint32_t tmem = pair_setup(s, warp);
    grid_dependency_wait();
    grid_launch_dependents();
    bool ok = true;
    // three warps share a scheduler's registers: 168 each at launch; the eight
    // epilogue warps, which hold 128 totals per thread, take what the others leave
    // (128 x 88 + 256 x 208 registers of 384 x 168)
    if (warp < kPairEpilogue) {
        regs_release<88>();
        if (warp == 0) ok = pair_produce<kMode, false, false, 128>(p.plan, maps, s, rank);
        if (warp == 1 && rank == 0) ok = pair_multiply<false, false, true, true>(p.plan, s, tmem);
        if (warp == 2) {
            uint32_t g = 0;
            for (int t = static_cast<int>(blockIdx.x >> 1); t < p.plan.ntiles; t += static_cast<int>(gridDim.x >> 1)) {
                const PairTileAt x = pair_tile(p.plan, t);
                const int m0 = x.mi * kPairTile + static_cast<int>(rank) * 128;
                for (int c = x.c0; c < x.c1; c += kScaleGroup, ++g) {
                    ScaleStage &st = scales[g & 1];
                    float w = 0.0f;   // lanes 0-7: the first weight block, 8-15: the second
                    {
                        const int second = lane >> 3, b = c + (lane & 7);
                        const int wb = kDual ? x.ni : 2 * x.ni + second;
                        if (second < 2 && b < x.c1 && wb < p.wblocks)
                            w = (kDual && second ? p.ws[1] + wb * p.ldws[1] : p.ws[0] + wb * p.ldws[0])[b];
                    }
                    if (g >= 2 && ok) ok = __all_sync(0xffffffffu, pair_wait(&scale_empty[g & 1], ((g >> 1) - 1) & 1, kWaitLimitNs));
#pragma unroll 1
                    for (int i0 = 0; i0 < 32; i0 += 16) {   // 4 rows x 8 blocks per load
                        float v[16];
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            const int m = m0 + 4 * (i0 + i) + (lane >> 3), b = c + (lane & 7);
                            v[i] = m < p.plan.rows && b < x.c1 ? p.as[m * p.ldas + b] : 0.0f;
                        }
#pragma unroll
                        for (int i = 0; i < 16; ++i) st.a[lane & 7][4 * (i0 + i) + (lane >> 3)] = v[i];
                    }
                    if (lane < 16) st.w[lane >> 3][lane & 7] = w;
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&scale_full[g & 1]);
                }
            }
        }
    } else {
        regs_take<208>();
        const int q = warp & 3, half = (warp - kPairEpilogue) >> 2;
        const uint32_t lanes = tmem + (static_cast<uint32_t>(q * 32) << 16);
        // this thread's accumulator columns: [col0, col0 + 64) and [col1, col1 + 64)
        const int col0 = kDual ? half * 64 : half * 128, col1 = kDual ? 128 + half * 64 : half * 128 + 64;
        uint32_t v = 0, tiles = 0, g = 0;
        for (int t = static_cast<int>(blockIdx.x >> 1); t < p.plan.ntiles; t += static_cast<int>(gridDim.x >> 1), ++tiles) {
            int c = 0, c1 = 0;
            {
                const PairTileAt x = pair_tile(p.plan, t);
                c = x.c0;
                c1 = x.c1;
            }
            const int first = c;
            uint64_t sums[64];   // pairs of columns
#pragma unroll
            for (int i = 0; i < 64; ++i) sums[i] = 0;
            // A step is 32 columns: its FMAs run while the next step's columns
            // arrive, over the blocks' borders too, so that tensor memory is read
            // without a pause (it gives a warp's 32 x 32 values in about 64 cycles:
            // 512 per block for the two warps of a scheduler, as long as the MMAs take).
            uint32_t r[2][32];
            if (ok) ok = pair_wait(&s.acc_full[v & 1], (v >> 1) & 1, kWaitLimitNs);
            __syncwarp();
            tc_fence_after();
            tmem_ld32(lanes + (v & 1) * kPairTile + static_cast<uint32_t>(col0), r[0]);
            tmem_wait_ld(r[0]);
#pragma unroll 1
            for (; c < c1; ++c, ++v) {
                const uint32_t buf = v & 1;
                const int in = (c - first) & (kScaleGroup - 1);
                if (in == 0 && ok) ok = pair_wait(&scale_full[g & 1], (g >> 1) & 1, kWaitLimitNs);
                const ScaleStage &sc = scales[g & 1];
                const float sa = sc.a[in][q * 32 + lane];
                const float s0 = sa * sc.w[kDual ? 0 : half][in], s1 = kDual ? sa * sc.w[1][in] : s0;
                const uint64_t f0 = pack_f32x2(s0, s0), f1 = kDual ? pack_f32x2(s1, s1) : f0;
                __syncwarp();
                if (in == kScaleGroup - 1 || c == c1 - 1) {   // the group is read
                    if (lane == 0) mbar_arrive(&scale_empty[g & 1]);
                    ++g;
                }
                const uint32_t from = lanes + buf * kPairTile;
#pragma unroll
                for (int j = 0; j < 3; ++j) {
                    tmem_ld32(from + static_cast<uint32_t>((j < 1 ? col0 : col1) + (~j & 1) * 32), r[(j + 1) & 1]);
                    const uint64_t f = j < 2 ? f0 : f1;
#pragma unroll
                    for (int i = 0; i < 16; ++i) scale_add(sums[16 * j + i], r[j & 1][2 * i], r[j & 1][2 * i + 1], f);
                    tmem_wait_ld(r[(j + 1) & 1]);
                }
                tc_fence_before();   // the buffer is read
                __syncwarp();
                if (lane == 0) pair_arrive(map_to_rank(&s.acc_empty[buf], 0));
                if (c + 1 < c1) {
                    if (ok) ok = pair_wait(&s.acc_full[buf ^ 1], ((v + 1) >> 1) & 1, kWaitLimitNs);
                    __syncwarp();
                    tc_fence_after();
                    tmem_ld32(lanes + (buf ^ 1) * kPairTile + static_cast<uint32_t>(col0), r[0]);
                }
#pragma unroll
                for (int i = 0; i < 16; ++i) scale_add(sums[48 + i], r[1][2 * i], r[1][2 * i + 1], f1);
                if (c + 1 < c1) tmem_wait_ld(r[0]);
            }
            // where the tile lies, worked out again: the loop above needs every register
            ok = __all_sync(0xffffffffu, ok);
            int again = t;
            asm volatile("" : "+r"(again));
            const PairTileAt x = pair_tile(p.plan, again);
            const int64_t m = static_cast<int64_t>(x.mi) * kPairTile + rank * 128 + q * 32;   // the warp's first row
            const int rows = static_cast<int>(min(static_cast<int64_t>(32), p.plan.rows - m));
            uint32_t *buf32 = s.row_bufs + (warp - kPairEpilogue) * kRowBuf;
            float2 acc[64];
#pragma unroll
            for (int i = 0; i < 64; ++i) acc[i] = unpack_f32x2(sums[i]);
            if constexpr (EPI == kFp8Out) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int n = x.ni * kPairTile + col0 + 32 * j, valid = p.plan.cols - n;
                    if (!ok || rows <= 0 || valid <= 0) continue;   // the whole warp
                    if (x.slot >= 0) {
                        uint32_t f[32];
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            f[2 * i] = __float_as_uint(acc[16 * j + i].x);
                            f[2 * i + 1] = __float_as_uint(acc[16 * j + i].y);
                        }
                        warp_store_f32(buf32, p.part + x.slot * kPairSlot + (rank * 128 + q * 32) * kPairTile + col0 + 32 * j, kPairTile, f,
                                       rows, 32, 2);
                    } else {
                        uint32_t w[16];
#pragma unroll
                        for (int i = 0; i < 16; ++i) w[i] = pack_bf16x2(acc[16 * j + i].x, acc[16 * j + i].y);
                        warp_store_bf16(buf32, p.out + m * p.ldo + n, p.ldo, w, rows, valid, p.out_align);
                    }
                }
            } else {
                // g in acc[0..31], u in acc[32..63]: SiLU(g) u over g
                const int n0 = x.ni * 128 + half * 64;
                float amax = 0.0f;
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                    acc[i].x = silu_short(acc[i].x) * acc[32 + i].x;
                    acc[i].y = silu_short(acc[i].y) * acc[32 + i].y;
                    // columns past the last are sums over zeros unless a scale is
                    // not finite; they are no part of the group
                    if (EPI == kFp8GluQuant) {
                        if (n0 + 2 * i < p.plan.cols) amax = max_nan(amax, fabsf(acc[i].x));
                        if (n0 + 2 * i + 1 < p.plan.cols) amax = max_nan(amax, fabsf(acc[i].y));
                    }
                }
                float scale = 0.0f, inv = 0.0f;
                if constexpr (EPI == kFp8GluQuant) {
                    // the other 64 columns' maximum, from the warp that has them
                    float *ex = s.exchange + (tiles & 1) * 256;
                    ex[half * 128 + q * 32 + lane] = amax;
                    bar_sync_named(1, 256);
                    amax = max_nan(amax, ex[(half ^ 1) * 128 + q * 32 + lane]);
                    scale = group_scale(amax);
                    inv = 1.0f / scale;
                    if (ok && lane < rows && half == 0) p.qs[(m + lane) * p.ldqs + x.ni] = scale;
                }
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int n = n0 + 32 * j, valid = p.plan.cols - n;
                    if (!ok || rows <= 0 || valid <= 0) continue;   // the whole warp
                    if constexpr (EPI == kFp8GluQuant) {
                        uint32_t w[8];
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const float2 a = acc[16 * j + 2 * i], b = acc[16 * j + 2 * i + 1];
                            w[i] = pack_e4m3x4(a.x * inv, a.y * inv, b.x * inv, b.y * inv);
                        }
                        warp_store_e4m3(buf32, p.q + m * p.ldq + n, p.ldq, w, rows, valid, p.q_align);
                    } else {
                        uint32_t w[16];
#pragma unroll
                        for (int i = 0; i < 16; ++i) w[i] = pack_bf16x2(acc[16 * j + i].x, acc[16 * j + i].y);
                        warp_store_bf16(buf32, p.out + m * p.ldo + n, p.ldo, w, rows, valid, p.out_align);
                    }
                }
            }
        }
    }
    if (!ok) atomicExch(&g_dense_error, kErrTimeout);
    pair_teardown(warp, tmem);
}

}  // namespace mbglu
