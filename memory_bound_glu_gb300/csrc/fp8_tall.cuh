// fp8_tall.cuh -- the e4m3 products of a token up to some dozens of rows (a
// decode step), and of any number of rows where the product has few tiles: too
// few to fill the 256-row side of a CTA pair's tile, or the part with such tiles.
// The weights take the MMA's 128-row side and the tokens its N, so that both the
// products and the reading of the accumulators shrink with the batch and what is
// left is the weights' bytes.
//
// More tokens than a tile holds are further tiles, which read the weights again,
// from L2.  Narrow tiles on more SMs are often the faster ones all the same (one
// weight of K = 4096, N = 1000 at M = 128: 6.1 us in tiles of 32 tokens, 8.9 in one
// of 128; K = 9728, N = 2560 at M = 333: 21.5 us in tiles of 112 and two ranges, 24.4
// on CTA pairs).  A stage of 128 tokens takes about 340 ns: 32 KB into every SM, 14.6
// TB/s in all, so L2 bounds what is not bound by a call's start and end.
//
// A block holds 128 weight rows -- one scale block, and one group of an e4m3
// output -- of one weight or of gate and up, TN tokens, and one of `ks` ranges
// of the inner dimension; the ranges of a tile are the blocks of a cluster.  Per
// 128 of the inner dimension (a scale block, a stage): one or two sums of
// 128 x TN in tensor memory, read by eight epilogue warps, scaled by the token's
// and the weight block's scale and added to fp32 totals in registers, while the
// next stage's sums are formed.  At the end each block gets the totals of its
// share of the tokens from all blocks of the cluster (distributed shared memory,
// added in rank order) and writes them.
//
// Roles (384 threads): warp 0 copies, warp 1 issues the MMAs and owns the tensor
// memory, warp 2 stages the scales, warps 4-11 are the epilogue: warp w has
// weight rows 32 (w % 4).. and half of the tokens.
#pragma once

#include "fp8_pair.cuh"

namespace mbglu {

constexpr int kTallRows = 128;
constexpr uint32_t kTallW = 16384;             // one weight's bytes per stage
constexpr int kTallMaxStages = 8;
constexpr uint32_t kTallHeader = 1024;
constexpr int kTallMaxSplit = 8;
constexpr int kTallGroup = 4;                  // scale blocks staged at a time

__host__ __device__ constexpr int tall_per_sm(int tn, bool dual) { return tn <= 16 || (dual && tn <= 32) ? 2 : 1; }

template <int TN, bool DUAL>
struct TallShape {
    static constexpr int kMats = DUAL ? 2 : 1;
    static constexpr uint32_t kStage = kMats * kTallW + TN * 128u;
    // the products of a token's and a weight's scale, of 4 blocks; two of them
    static constexpr uint32_t kScales = kMats * TN * kTallGroup * 4u;
    // Small sums leave registers and tensor memory for two blocks per SM: one
    // block's start and end then lie under another's stream, and the next call's
    // first weights under this call's last (two weights of K = 4096, N = 11008,
    // chained: 18.0 us against 22.3 at M = 16, 21.3 against 26.1 at M = 32; one
    // weight at M = 32: 8.8 against 8.4, so not there).
    static constexpr int kPerSm = tall_per_sm(TN, DUAL);
    static constexpr uint32_t kRoom = (kPerSm == 2 ? 113u : 225u) * 1024 - 1024 - kTallHeader - 2 * kScales;
    static constexpr int kStages = kRoom / kStage < kTallMaxStages ? static_cast<int>(kRoom / kStage) : kTallMaxStages;
    static constexpr uint32_t kSmem = 1024 + kTallHeader + 2 * kScales + kStages * kStage;
    // the totals that a block gets: every rank's, of its share of the tokens
    static constexpr uint32_t totals(int ks) { return static_cast<uint32_t>(ks * kMats * ((TN + ks - 1) / ks)) * kTallRows * 4u; }
    // tensor-memory columns of one of the two buffers
    static constexpr uint32_t cols(uint32_t n) { return n <= 16 ? 16 : n <= 32 ? 32 : n <= 64 ? 64 : n <= 128 ? 128 : 256; }
    static constexpr uint32_t kCols = cols(kMats * TN);
    static_assert(totals(1) <= kStages * kStage && totals(3) <= kStages * kStage && totals(5) <= kStages * kStage &&
                      totals(6) <= kStages * kStage && totals(7) <= kStages * kStage,
                  "the exchange fits the stages");
    static_assert(kStages >= 3 && kSmem <= 227u * 1024, "shared memory");
};

struct TallMaps {
    TensorMap w[2], x;
};

struct TallParams {
    int M, N, nchunk, ks, wtiles;
    int prefetch;
    const float *as;
    int64_t ldas;
    const float *ws[2];
    int64_t ldws[2];
    uint16_t *out;
    int64_t ldo;
    uint8_t *q;
    int64_t ldq;
    float *qs;
    int64_t ldqs;
};

__device__ __forceinline__ void tc_mma_e4m3(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc, bool accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(static_cast<uint32_t>(accumulate))
        : "memory");
}

// OUT: 0 bf16 product (one weight), 1 bf16 gated, 2 e4m3 gated.
template <int TN, int OUT>
__global__ void __launch_bounds__(384, tall_per_sm(TN, OUT != 0)) fp8_tall_kernel(const TallParams p, const __grid_constant__ TallMaps maps)
{
    constexpr bool kDual = OUT != 0;
    using Shape = TallShape<TN, kDual>;
    constexpr int kMats = Shape::kMats, kStages = Shape::kStages;
    constexpr int TH = TN / 2;                     // tokens per thread
    constexpr int SW = TH % 32 == 0 ? 32 : TH % 16 == 0 ? 16 : 8;   // columns per step
    constexpr int kSteps = TH / SW;                // steps per matrix
    extern __shared__ unsigned char tall_raw[];
    unsigned char *base = tall_raw + ((1024u - (smem_addr(tall_raw) & 1023u)) & 1023u);
    uint64_t *full = reinterpret_cast<uint64_t *>(base);
    uint64_t *empty = full + kTallMaxStages, *acc_full = empty + kTallMaxStages, *acc_empty = acc_full + 2;
    uint64_t *scale_full = acc_empty + 2, *scale_empty = scale_full + 2;
    uint32_t *slot = reinterpret_cast<uint32_t *>(scale_empty + 2);
    float *peaks = reinterpret_cast<float *>(base + 512);   // 2 x 8 warps x 8 tokens
    unsigned char *stages = base + kTallHeader;
    float *scales = reinterpret_cast<float *>(stages + kStages * Shape::kStage);
    constexpr int kScaleFloats = Shape::kScales / 4;
    float *totals = reinterpret_cast<float *>(stages);      // after the products: [rank][mat][token][128 rows]

    const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
    const int ks = p.ks;
    const int rank = ks > 1 ? static_cast<int>(cluster_ctarank()) : 0;
    const int unit = static_cast<int>(blockIdx.x) / ks;
    const int wt = unit % p.wtiles, m0 = unit / p.wtiles * TN;
    const int c0 = p.nchunk * rank / ks, c1 = p.nchunk * (rank + 1) / ks;

    if (threadIdx.x == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&acc_full[i], 1);
            mbar_init(&acc_empty[i], 8);
            mbar_init(&scale_full[i], 1);
            mbar_init(&scale_empty[i], 8);
        }
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc(slot, 2 * Shape::kCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    __syncwarp();
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xffffffffu, *slot, 0);
    bool ok = true;
    // the copies of the weights may start before the preceding kernel has ended;
    // everything else waits for it
    if (warp != 0 || !p.prefetch) grid_dependency_wait();
    if (warp != 0) grid_launch_dependents();

    if (warp < 4) {
        if (Shape::kPerSm == 1) regs_release<88>();
        if (warp == 0) {
            auto load_w = [&](int st, int c) {
                unsigned char *d = stages + st * Shape::kStage;
                mbar_arrive_expect_tx(&full[st], Shape::kStage);
#pragma unroll
                for (int i = 0; i < kMats; ++i)
                    tma_load_2d(d + i * kTallW, &maps.w[i], c * 128, wt * kTallRows, &full[st], l2_policy_evict_first());
            };
            auto load_x = [&](int st, int c) {
                tma_load_2d(stages + st * Shape::kStage + kMats * kTallW, &maps.x, c * 128, m0, &full[st], l2_policy_evict_last());
            };
            const int early = p.prefetch ? min(kStages, c1 - c0) : 0;
            if (early > 0) {
                if (elect_one())
                    for (int i = 0; i < early; ++i) load_w(i, c0 + i);
                __syncwarp();
                grid_dependency_wait();
                if (elect_one())
                    for (int i = 0; i < early; ++i) load_x(i, c0 + i);
                __syncwarp();
            } else if (p.prefetch) {
                grid_dependency_wait();
            }
            grid_launch_dependents();
            int st = early == kStages ? 0 : early;
            uint32_t phase = early == kStages ? 0 : 1;
            int filled = early;
            for (int c = c0 + early; c < c1; ++c) {
                if (!pair_wait(&empty[st], phase, kWaitLimitNs)) {
                    ok = false;
                    break;
                }
                __syncwarp();
                if (elect_one()) {
                    load_w(st, c);
                    load_x(st, c);
                }
                __syncwarp();
                if (filled < kStages) ++filled;
                if (++st == kStages) {
                    st = 0;
                    phase ^= 1;
                }
            }
            // every copy has landed and been read before the stages take the totals
            for (int i = 0; i < filled; ++i) {
                int at = st - (filled - i);
                const uint32_t ph = at < 0 ? phase : phase ^ 1;   // filled in the round before this one, or in this
                if (at < 0) at += kStages;
                if (!pair_wait(&empty[at], ph, kWaitLimitNs)) ok = false;
            }
            __syncwarp();
        } else if (warp == 1) {
            constexpr uint32_t idesc = (1u << 4) | (static_cast<uint32_t>(TN >> 3) << 17) | (static_cast<uint32_t>(kTallRows >> 4) << 24);
            const uint64_t d0 = smem_desc_sw128(stages);
            int st = 0;
            uint32_t phase = 0, buf = 0, acc_phase = 1;
            for (int c = c0; c < c1 && ok; ++c) {
                ok = pair_wait(&acc_empty[buf], acc_phase, kWaitLimitNs) && pair_wait(&full[st], phase, kWaitLimitNs);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                tc_fence_after();
                const uint64_t w = d0 + static_cast<uint32_t>(st) * (Shape::kStage >> 4);
                const uint64_t x = w + kMats * (kTallW >> 4);
                const uint32_t d = tmem + buf * Shape::kCols;
                if (elect_one()) {
#pragma unroll
                    for (int i = 0; i < kMats; ++i)
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)
                            tc_mma_e4m3(d + i * TN, w + i * (kTallW >> 4) + 2 * kk, x + 2 * kk, idesc, kk > 0);
                    tc_commit(&empty[st]);
                    tc_commit(&acc_full[buf]);
                }
                __syncwarp();
                if (++st == kStages) {
                    st = 0;
                    phase ^= 1;
                }
                buf ^= 1;
                if (buf == 0) acc_phase ^= 1;
            }
        } else if (warp == 2) {
            uint32_t g = 0;
            for (int c = c0; c < c1; c += kTallGroup, ++g) {
                float *sc = scales + (g & 1) * kScaleFloats;
                const int in = lane & 3, b = c + in;
                float w[kMats];
#pragma unroll
                for (int d = 0; d < kMats; ++d) w[d] = b < c1 ? p.ws[d][wt * p.ldws[d] + b] : 0.0f;
                if (g >= 2 && ok) ok = __all_sync(0xffffffffu, pair_wait(&scale_empty[g & 1], ((g >> 1) - 1) & 1, kWaitLimitNs));
#pragma unroll 8
                for (int i = 0; i < TN / 8; ++i) {   // 8 tokens x 4 blocks per load
                    const int tok = 8 * i + (lane >> 2), m = m0 + tok;
                    const float x = m < p.M && b < c1 ? p.as[m * p.ldas + b] : 0.0f;
#pragma unroll
                    for (int d = 0; d < kMats; ++d) sc[(d * kTallGroup + in) * TN + tok] = x * w[d];
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&scale_full[g & 1]);
            }
        }
        __syncwarp();
        if (ks > 1) cluster_sync();   // every block's products are done: the stages are free
        else __syncthreads();
        if (ks > 1) cluster_sync();   // the totals have come
        else __syncthreads();
    } else {
        if (Shape::kPerSm == 1) regs_take<208>();
        const int q = warp & 3, half = (warp - 4) >> 2;
        const uint32_t lanes = tmem + (static_cast<uint32_t>(q * 32) << 16) + static_cast<uint32_t>(half * TH);
        const int row = q * 32 + lane;
        uint64_t sums[kMats][TH / 2];
#pragma unroll
        for (int d = 0; d < kMats; ++d)
#pragma unroll
            for (int i = 0; i < TH / 2; ++i) sums[d][i] = 0;
        uint32_t v = 0, g = 0;
        if (c0 < c1) {
            uint32_t r[2][SW];
            if (ok) ok = pair_wait(&acc_full[0], 0, kWaitLimitNs);
            __syncwarp();
            tc_fence_after();
            tmem_load(lanes, r[0]);
            tmem_wait_ld(r[0]);
#pragma unroll 1
            for (int c = c0; c < c1; ++c, ++v) {
                const uint32_t buf = v & 1;
                const int in = (c - c0) & (kTallGroup - 1);
                if (in == 0 && ok) ok = pair_wait(&scale_full[g & 1], (g >> 1) & 1, kWaitLimitNs);
                __syncwarp();
                const float *sc = scales + (g & 1) * kScaleFloats;
                const float *sx = sc + in * TN + half * TH;
                const uint32_t from = lanes + buf * Shape::kCols;
#pragma unroll
                for (int s = 0; s < kMats * kSteps; ++s) {
                    const int next = s + 1;
                    if (next < kMats * kSteps) {
                        tmem_load(from + static_cast<uint32_t>(next / kSteps * TN + next % kSteps * SW), r[next & 1]);
                    } else {
                        tc_fence_before();   // the buffer is read
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&acc_empty[buf]);
                        if (c + 1 < c1) {
                            if (ok) ok = pair_wait(&acc_full[buf ^ 1], ((v + 1) >> 1) & 1, kWaitLimitNs);
                            __syncwarp();
                            tc_fence_after();
                            tmem_load(lanes + (buf ^ 1) * Shape::kCols, r[next & 1]);
                        }
                    }
                    const int d = s / kSteps, t0 = s % kSteps * SW;
#pragma unroll
                    for (int i = 0; i < SW / 4; ++i) {
                        const float4 f = *reinterpret_cast<const float4 *>(sx + d * kTallGroup * TN + t0 + 4 * i);
                        scale_add(sums[d][t0 / 2 + 2 * i], r[s & 1][4 * i], r[s & 1][4 * i + 1], pack_f32x2(f.x, f.y));
                        scale_add(sums[d][t0 / 2 + 2 * i + 1], r[s & 1][4 * i + 2], r[s & 1][4 * i + 3], pack_f32x2(f.z, f.w));
                    }
                    if (next < kMats * kSteps || c + 1 < c1) tmem_wait_ld(r[next & 1]);
                }
                if (kMats * kSteps % 2 == 1) {   // an odd number of steps: the next block's first columns are in r[1]
#pragma unroll
                    for (int i = 0; i < SW; ++i) r[0][i] = r[1][i];
                }
                if (in == kTallGroup - 1 || c == c1 - 1) {   // the scales are read
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&scale_empty[g & 1]);
                    ++g;
                }
            }
        }
        ok = __all_sync(0xffffffffu, ok);
        // each token's totals to the block that writes it
        const int share = (TN + ks - 1) / ks;
        if (ks > 1) cluster_sync();
        else __syncthreads();
        fence_proxy_async_smem();
        {
            int owner = half * TH / share, tok = half * TH - owner * share;
            uint32_t dst = map_to_rank(totals, static_cast<uint32_t>(owner));
#pragma unroll
            for (int i = 0; i < TH; ++i) {
                const int at = (rank * kMats * share + tok) * kTallRows + row;
#pragma unroll
                for (int d = 0; d < kMats; ++d) {
                    const float2 x = unpack_f32x2(sums[d][i / 2]);
                    st_cluster_f32(dst + static_cast<uint32_t>(at + d * share * kTallRows) * 4u, i & 1 ? x.y : x.x);
                }
                if (++tok == share) {
                    tok = 0;
                    ++owner;
                    if (i + 1 < TH) dst = map_to_rank(totals, static_cast<uint32_t>(min(owner, ks - 1)));
                }
            }
        }
        if (ks > 1) cluster_sync();
        else __syncthreads();
        // this block's tokens: warps 4-7 and 8-11 take groups of kGroup in turn (as many
        // chains of loads, SiLUs and shuffles at once), a thread one weight row.  A tile
        // of few tokens has small groups: code that runs once is bound by its fetching
        // (one weight of K = 9728, N = 2560 at M = 8: 7.0 us with groups of one, 7.6 of
        // four; two of K = 4096, N = 11008 in tiles of 64 tokens: 27.0 with eight, 29.8 with four).
        constexpr int kGroup = TN <= 16 ? (OUT == 0 ? 1 : 2) : TN <= 32 && OUT == 0 ? 4 : 8;
        const int n = wt * kTallRows + row;
        const int first = rank * share, count = min(min(share, TN - first), p.M - m0 - first);
        for (int g0 = 0; g0 < count; g0 += 2 * kGroup) {   // both halves run the same rounds: there is a barrier
            const int t0 = g0 + half * kGroup;
            float val[kGroup], up[kGroup];
#pragma unroll
            for (int u = 0; u < kGroup; ++u) val[u] = up[u] = 0.0f;
            const float *from = totals + t0 * kTallRows + row;
            for (int s = 0; s < ks; ++s, from += kMats * share * kTallRows) {
#pragma unroll
                for (int u = 0; u < kGroup; ++u) {
                    if (t0 + u >= count) break;
                    val[u] += from[u * kTallRows];
                    if (kDual) up[u] += from[(share + u) * kTallRows];
                }
            }
            if (kDual) {
#pragma unroll
                for (int u = 0; u < kGroup; ++u) val[u] = silu_short(val[u]) * up[u];
            }
            const int64_t m = m0 + first + t0;
            if constexpr (OUT == 2) {
                float amax[kGroup];
#pragma unroll
                for (int u = 0; u < kGroup; ++u) amax[u] = n < p.N ? fabsf(val[u]) : 0.0f;
#pragma unroll
                for (int o = 16; o > 0; o >>= 1)
#pragma unroll
                    for (int u = 0; u < kGroup; ++u) amax[u] = max_nan(amax[u], __shfl_xor_sync(0xffffffffu, amax[u], o));
                // the four warps of a half hold the group; two sets of places, used in turn
                float *pk = peaks + ((g0 / (2 * kGroup)) & 1) * 8 * kGroup + half * 4 * kGroup;
                if (lane == 0) {
#pragma unroll
                    for (int u = 0; u < kGroup; ++u) pk[q * kGroup + u] = amax[u];
                }
                bar_sync_named(1, 256);
#pragma unroll
                for (int u = 0; u < kGroup; ++u) {
                    const float a = max_nan(max_nan(pk[u], pk[kGroup + u]), max_nan(pk[2 * kGroup + u], pk[3 * kGroup + u]));
                    const float s = group_scale(a);
                    if (t0 + u < count && ok) {
                        if (row == 0) p.qs[(m + u) * p.ldqs + wt] = s;
                        if (n < p.N) p.q[(m + u) * p.ldq + n] = static_cast<uint8_t>(pack_e4m3x2(val[u] * (1.0f / s), 0.0f));
                    }
                }
            } else {
#pragma unroll
                for (int u = 0; u < kGroup; ++u)
                    if (t0 + u < count && ok && n < p.N) p.out[(m + u) * p.ldo + n] = f32_to_bf16(val[u]);
            }
        }
    }
    if (!ok) atomicExch(&g_dense_error, kErrTimeout);
    tc_fence_before();
    __syncthreads();
    __syncwarp();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, 2 * Shape::kCols);
    }
}

}  // namespace mbglu
