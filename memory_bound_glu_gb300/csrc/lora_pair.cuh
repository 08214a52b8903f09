// lora_pair.cuh -- products with low-rank adapters on CTA pairs: the shared product with
// the weights on the MMA's 256-row side and the tokens on the other (pair_tall.cuh's
// tiles and roles), and the adapters' term added where the accumulators are read.
//
// The adapters' term p[m] B[a]^T is not a product of matrices: every row has a B of its
// own.  Tokens are taken eight at a time: for each adapter among them a warp's tensor
// cores multiply its 32 rows of B with the eight tokens' p (as two bf16 terms, off by
// 2^-18), and a token takes the product with its own adapter.  So nothing of other adapters
// enters a token's sum, infinities neither, and eight tokens of one adapter cost one such
// product.
//
// Tiles that would leave SM pairs without work are cut along the inner dimension: their
// ranges leave partial sums, and lora_join_kernel adds them, the adapters' term and the
// epilogue.  There a lane has one output and reads its row of B, the term in fp32 FMAs.
#pragma once
#include "lora_shrink.cuh"
#include "pair_gemm.cuh"

namespace mbglu {

struct LoraPlan {
    int tn, wt;              // tokens and outputs per tile
    int ttiles, ntiles;      // tiles along the tokens, in all
    int whole;               // tiles done whole
    int rest, splits;        // the others, each in `splits` ranges of the inner dimension
    int items;               // whole + rest splits
    int nchunk;
};

struct LoraPairParams {
    LoraParams l;
    LoraPlan plan;
    float *part;             // [rest splits][tn][256]: a range's accumulators, token by token
    int early;               // the kernel before this one has waited for the operands
};

struct LoraTile {
    int t, c0, c1, slot;     // tile, chunks, where a range's sums go or -1
};

__host__ __device__ inline LoraTile lora_tile(const LoraPlan &p, int i)
{
    LoraTile x;
    x.slot = i < p.whole ? -1 : i - p.whole;
    x.t = i;
    x.c0 = 0;
    x.c1 = p.nchunk;
    if (x.slot >= 0) {
        const int split = x.slot / p.rest;
        x.t = p.whole + x.slot % p.rest;
        x.c0 = static_cast<int>(static_cast<int64_t>(p.nchunk) * split / p.splits);
        x.c1 = static_cast<int>(static_cast<int64_t>(p.nchunk) * (split + 1) / p.splits);
    }
    return x;
}

// The adapters' term of 32 outputs from n0 on and eight tokens from m0 on: term[token *
// kTermPitch + output].  The whole warp; whether there was any is returned.
constexpr int kTermPitch = 36;
constexpr int kTermWords = 8 * kTermPitch;
__device__ __forceinline__ bool lora_term(const LoraParams &p, int d, int sides, int64_t m0, int n0, float *term)
{
    const int lane = threadIdx.x & 31, row = lane >> 2, quad = lane & 3;
    const int64_t m = m0 + row;
    const int mine = lora_adapter(p, m);
    uint32_t left = __ballot_sync(0xffffffffu, mine >= 0);
    if (!left) return false;
    const LoraSide &side = p.side[d];
    const float *q = p.p + m * sides * p.R + d * p.R + quad * 4;
    float sum[2][4] = {};
    while (left) {
        const int a = __shfl_sync(0xffffffffu, mine, __ffs(left) - 1);
        const uint32_t match = __ballot_sync(0xffffffffu, mine == a);
        left &= ~match;
        float acc[2][4] = {};
        const uint16_t *b = side.b + a * side.b_adapter + (n0 + row) * side.ldb + quad * 4;
#pragma unroll 2
        for (int j = 0; j < p.R; j += 16) {
            const bool in = j + quad * 4 < p.R;
            uint2 w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                w[i] = in && n0 + row + i * 8 < p.N ? *reinterpret_cast<const uint2 *>(b + i * 8 * side.ldb + j) : make_uint2(0, 0);
            const float4 v = in && mine >= 0 ? *reinterpret_cast<const float4 *>(q + j) : make_float4(0, 0, 0, 0);
            const uint32_t h0 = pack_bf16x2(v.x, v.y), h1 = pack_bf16x2(v.z, v.w);
            const uint32_t l0 = pack_bf16x2(v.x - bf16_lo(h0), v.y - bf16_hi(h0)), l1 = pack_bf16x2(v.z - bf16_lo(h1), v.w - bf16_hi(h1));
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                const uint32_t wa[4] = {w[2 * t].x, w[2 * t + 1].x, w[2 * t].y, w[2 * t + 1].y};
                mma_16816(acc[t], wa, h0, h1);
                mma_16816(acc[t], wa, l0, l1);
            }
        }
        // this lane's two tokens: quad * 2 and the next; a token's four lanes vote alike
        const bool t0 = match >> (quad * 8) & 1u, t1 = match >> (quad * 8 + 4) & 1u;
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            sum[t][0] = t0 ? acc[t][0] : sum[t][0];
            sum[t][1] = t1 ? acc[t][1] : sum[t][1];
            sum[t][2] = t0 ? acc[t][2] : sum[t][2];
            sum[t][3] = t1 ? acc[t][3] : sum[t][3];
        }
    }
    __syncwarp();
#pragma unroll
    for (int t = 0; t < 2; ++t) {
        float *o = term + quad * 2 * kTermPitch + t * 16 + row;
        o[0] = sum[t][0];
        o[kTermPitch] = sum[t][1];
        o[8] = sum[t][2];
        o[kTermPitch + 8] = sum[t][3];
    }
    __syncwarp();
    return true;
}

// The exchange between the two warps of an output's g and u (as pair_tall.cuh), then the
// warps' terms.
constexpr int kLoraSwap = 2 * 16 * 32;
constexpr uint32_t kLoraExtra = 4 * kLoraSwap * 4 + 8 * kTermWords * 4;
constexpr uint32_t kLoraSmem = kPairHeader + kPairStages * kPairStage + kLoraExtra + 1024;
static_assert(kLoraSmem <= 227 * 1024, "shared memory");

template <int SIDES>
__global__ void __launch_bounds__(kPairThreads, 1) lora_pair_kernel(const LoraPairParams p, const __grid_constant__ PairMaps maps)
{
    extern __shared__ unsigned char pair_raw[];
    const PairShared s = pair_shared(pair_raw);
    const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
    const int rank = static_cast<int>(cluster_ctarank());
    const uint32_t tmem = pair_setup(s, warp);
    const LoraPlan &plan = p.plan;
    bool ok = true;
    const int first = static_cast<int>(blockIdx.x >> 1), step = static_cast<int>(gridDim.x >> 1);
    if (!p.early) grid_dependency_wait();
    grid_launch_dependents();

    if (warp == 0) {
        const uint32_t full0 = map_to_rank(s.full, 0);
        // both CTAs'; of one projection a CTA's rows are one box
        const uint32_t bytes = static_cast<uint32_t>(plan.wt) * (SIDES == 2 ? 256u : 128u) + static_cast<uint32_t>(plan.tn) * 128u;
        int st = 0, filled = 0;
        uint32_t phase = 1;
        for (int i = first; i < plan.items && ok; i += step) {
            const LoraTile x = lora_tile(plan, i);
            const int n0 = x.t / plan.ttiles * plan.wt + rank * (plan.wt / 2), m0 = x.t % plan.ttiles * plan.tn + rank * (plan.tn / 2);
            for (int c = x.c0; c < x.c1; ++c) {
                if (!pair_wait(&s.empty[st], phase, kWaitLimitNs)) {
                    ok = false;
                    break;
                }
                unsigned char *d = s.stages + st * kPairStage;
                const uint32_t bar = full0 + static_cast<uint32_t>(st) * 8u;
                if (elect_one()) {
                    if (rank == 0) mbar_arrive_expect_tx(&s.full[st], bytes);
                    pair_load_2d(d, &maps.a[0], c * 64, n0, bar);
                    if (SIDES == 2) pair_load_2d(d + kPairOperand / 2, &maps.a[1], c * 64, n0, bar);
                    pair_load_2d(d + kPairOperand, &maps.b[0], c * 64, m0, bar);
                }
                __syncwarp();
                filled += filled < kPairStages;
                if (++st == kPairStages) {
                    st = 0;
                    phase ^= 1;
                }
            }
        }
        for (int i = 0; i < filled; ++i) {   // as pair_produce: the last round's stages, oldest first
            int at = st - (filled - i);
            const uint32_t ph = at < 0 ? phase : phase ^ 1;
            if (at < 0) at += kPairStages;
            if (!pair_wait(&s.empty[at], ph, kWaitLimitNs)) ok = false;
        }
    } else if (warp == 1) {
        if (rank == 0) {
            const uint32_t idesc = tc_idesc_bf16(256, 256) - (static_cast<uint32_t>((256 - plan.tn) >> 3) << 17);
            const uint64_t a0 = smem_desc_sw128(s.stages), b0 = smem_desc_sw128(s.stages + kPairOperand);
            int st = 0;
            uint32_t phase = 0, buf = 0, acc_phase = 1;
            for (int i = first; i < plan.items && ok; i += step) {
                const LoraTile x = lora_tile(plan, i);
                for (int c = x.c0; c < x.c1; ++c) {
                    if ((c == x.c0 && !pair_wait(&s.acc_empty[buf], acc_phase, kWaitLimitNs)) || !pair_wait(&s.full[st], phase, kWaitLimitNs)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint64_t a = a0 + static_cast<uint32_t>(st) * (kPairStage >> 4), b = b0 + static_cast<uint32_t>(st) * (kPairStage >> 4);
                    if (elect_one()) {
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk) pair_mma_bf16(tmem + buf * kPairTile, a + 2 * kk, b + 2 * kk, idesc, kk > 0 || c > x.c0);
                        pair_commit(&s.empty[st]);
                        if (c == x.c1 - 1) pair_commit(&s.acc_full[buf]);
                    }
                    __syncwarp();
                    if (++st == kPairStages) {
                        st = 0;
                        phase ^= 1;
                    }
                }
                buf ^= 1;
                if (buf == 0) acc_phase ^= 1;
            }
        }
    } else if (warp >= kPairEpilogue) {
        // p, and what the join reads after this kernel, come from the kernel before
        if (p.early) grid_dependency_wait();
        const int q = warp & 3, half = (warp - kPairEpilogue) >> 2, d = SIDES == 2 ? q >> 1 : 0;
        const uint32_t lanes = tmem + (static_cast<uint32_t>(q * 32) << 16) + static_cast<uint32_t>(half * (plan.tn / 2));
        const int pairing = half * 2 + (q & 1);
        float *extra = reinterpret_cast<float *>(s.row_bufs);
        float *swap = extra + pairing * kLoraSwap + lane, *term = extra + 4 * kLoraSwap + (warp - kPairEpilogue) * kTermWords;
        const int row0 = SIDES == 2 ? (q & 1) * 32 : q * 32;   // the warp's first output of the CTA's
        uint32_t v = 0, sets = 0;
        for (int i = first; i < plan.items; i += step, ++v) {
            const LoraTile x = lora_tile(plan, i);
            const uint32_t buf = v & 1;
            const int n0 = x.t / plan.ttiles * plan.wt + rank * (plan.wt / 2) + row0;
            const int n = row0 + lane < plan.wt / 2 ? n0 + lane : p.l.N;   // N: none
            const int m0 = x.t % plan.ttiles * plan.tn + half * (plan.tn / 2);
            if (ok) ok = __all_sync(0xffffffffu, pair_wait(&s.acc_full[buf], (v >> 1) & 1, kWaitLimitNs));
            tc_fence_after();
            for (int j = 0; j < plan.tn / 2; j += 16, ++sets) {
                uint32_t r[16];
                __syncwarp();
                tmem_load(lanes + buf * kPairTile + static_cast<uint32_t>(j), r);
                tmem_wait_ld(r);
                if (j + 16 == plan.tn / 2) {   // the buffer is read
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) pair_arrive(map_to_rank(&s.acc_empty[buf], 0));
                }
                const int tokens = ok ? p.l.M - m0 - j : 0;
                if (x.slot >= 0) {
                    float *o = p.part + (static_cast<int64_t>(x.slot) * plan.tn + half * (plan.tn / 2) + j) * 256 + rank * 128 + q * 32 + lane;
#pragma unroll
                    for (int k = 0; k < 16; ++k)
                        if (k < tokens) __stcg(o + k * 256, __uint_as_float(r[k]));
                    continue;   // the whole tile, in every warp: no exchange is begun
                }
                float y[16];
#pragma unroll
                for (int k = 0; k < 16; ++k) y[k] = __uint_as_float(r[k]);
#pragma unroll
                for (int g = 0; g < 2; ++g)
                    if (g * 8 < tokens && p.l.adapters > 0 && lora_term(p.l, d, SIDES, static_cast<int64_t>(m0) + j + g * 8, n0, term)) {
#pragma unroll
                        for (int k = 0; k < 8; ++k) y[g * 8 + k] += term[k * kTermPitch + lane];
                    }
                if constexpr (SIDES == 2) {
                    // two sets in turn, as in pair_tall_kernel
                    float *mine = swap + (sets & 1) * 512 + d * 256, *theirs = swap + (sets & 1) * 512 + (d ^ 1) * 256;
#pragma unroll
                    for (int k = 0; k < 8; ++k) mine[k * 32] = d ? y[k] : y[8 + k];
                    bar_sync_named(1 + pairing, 64);
                    const int m = m0 + j + d * 8, left = n < p.l.N && ok ? p.l.M - m : 0;
                    uint16_t *o = p.l.out + static_cast<int64_t>(m) * p.l.ldo + n;
                    uint16_t z[8];
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        const float other = theirs[k * 32], own = d ? y[8 + k] : y[k];
                        const float g = d ? other : own, u = d ? own : other;
                        z[k] = p.l.mode == 0 ? f32_to_bf16(silu_short(g) * u) : static_cast<uint16_t>(glu_hf_short(g, u));
                    }
#pragma unroll
                    for (int k = 0; k < 8; ++k, o += p.l.ldo)
                        if (k < left) *o = z[k];
                } else {
                    const int left = n < p.l.N ? tokens : 0;
                    uint16_t *o = p.l.out + static_cast<int64_t>(m0 + j) * p.l.ldo + n;
#pragma unroll
                    for (int k = 0; k < 16; ++k, o += p.l.ldo)
                        if (k < left) *o = f32_to_bf16(y[k]);
                }
            }
        }
    }
    if (!ok) atomicExch(&g_dense_error, kErrTimeout);
    pair_teardown(warp, tmem);
}

// The tiles in ranges: their partial sums in order, the adapters' term and the epilogue.  A
// warp takes 32 outputs and four tokens.
template <int SIDES>
__global__ void __launch_bounds__(256) lora_join_kernel(const LoraPairParams p)
{
    grid_dependency_wait();
    grid_launch_dependents();
    const LoraPlan &plan = p.plan;
    const int lane = threadIdx.x & 31;
    const int groups = plan.tn / 4, blocks = (plan.wt + 31) / 32;   // of a tile
    const int64_t total = static_cast<int64_t>(plan.rest) * blocks * groups;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5); i < total; i += static_cast<int64_t>(gridDim.x) * 8) {
        const int tile = static_cast<int>(i / (blocks * groups)), rest = static_cast<int>(i % (blocks * groups));
        const int t = plan.whole + tile, j0 = rest % groups * 4, w = rest / groups * 32 + lane;
        const int n = t / plan.ttiles * plan.wt + w;
        const int64_t m0 = static_cast<int64_t>(t % plan.ttiles) * plan.tn + j0;
        const int tokens = static_cast<int>(min(static_cast<int64_t>(4), p.l.M - m0));
        if (tokens <= 0 || w >= plan.wt || n >= p.l.N) continue;
        // output w of the tile: a CTA holds wt / 2 of them, in dual tiles from lanes 0 and 64 on
        const int rank = w >= plan.wt / 2 ? 1 : 0, at = rank * 128 + w - rank * (plan.wt / 2);
        float acc[4][SIDES] = {};
        for (int s = 0; s < plan.splits; ++s) {
            const float *q = p.part + ((static_cast<int64_t>(s) * plan.rest + tile) * plan.tn + j0) * 256 + at;
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (k < tokens) {
#pragma unroll
                    for (int d = 0; d < SIDES; ++d) acc[k][d] += __ldcg(q + k * 256 + d * 64);
                }
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if (k >= tokens) break;
            const int64_t m = m0 + k;
            const int a = lora_adapter(p.l, m);
            if (a >= 0) {
#pragma unroll
                for (int d = 0; d < SIDES; ++d) {
                    const LoraSide &side = p.l.side[d];
                    const uint16_t *b = side.b + a * side.b_adapter + n * side.ldb;
                    const float *v = p.l.p + m * SIDES * p.l.R + d * p.l.R;
                    float sum = 0.0f;
#pragma unroll 4
                    for (int j = 0; j < p.l.R; j += 4) {
                        const uint2 x = *reinterpret_cast<const uint2 *>(b + j);
                        const float4 y = *reinterpret_cast<const float4 *>(v + j);
                        sum = fmaf(bf16_lo(x.x), y.x, sum);
                        sum = fmaf(bf16_hi(x.x), y.y, sum);
                        sum = fmaf(bf16_lo(x.y), y.z, sum);
                        sum = fmaf(bf16_hi(x.y), y.w, sum);
                    }
                    acc[k][d] += sum;
                }
            }
            uint16_t *o = p.l.out + m * p.l.ldo + n;
            if constexpr (SIDES == 2)
                *o = p.l.mode == 0 ? f32_to_bf16(silu_short(acc[k][0]) * acc[k][SIDES - 1]) : static_cast<uint16_t>(glu_hf_short(acc[k][0], acc[k][SIDES - 1]));
            else
                *o = f32_to_bf16(acc[k][0]);
        }
    }
}

}  // namespace mbglu
