// lora_pair.cuh -- products with low-rank adapters on CTA pairs: the shared product with
// the weights on the MMA's 256-row side and the tokens on the other (pair_tall.cuh's
// tiles and roles), and the adapters' term added where the accumulators are read.
//
// The adapters' term p[m] B[a]^T is not a product of matrices: every row has a B of its
// own, and what another row's adapter holds, infinities too, must not reach it.  So:
//   * 32 rows of one adapter, and runs of them, go through the tensor cores as the shared
//     product does: more chunks of the inner dimension, with B as the weights and p's two
//     bf16 terms (off by 2^-18) as the tokens, into the run's columns of the accumulator.
//     With two projections the inner dimension is p = [gate's | up's]; a box of B that
//     begins R columns early, or ends late, is filled with zeros there.
//   * 32 rows of several adapters are left to the epilogue: for each adapter among 16 of
//     them a warp's own tensor cores (mma.sync) multiply its 32 rows of B with all 16
//     tokens' p, and a token takes the product with its own adapter (lora_term); up to rank
//     16, and in a decode batch, a lane reads the row of B of its output for each token
//     (lora_term_rows).
// A prompt's rows are nearly all of the first kind, a chunk of many short requests has the
// second.
//
// For most batches up to 320 rows no kernel of its own forms p: the epilogue's warps do, while
// the products run (lora_dot8).  Where the join uses p, the blocks share the work; where a block needs it itself
// and it is small (a token or some), every block forms all of it from L2.
//
// Tiles that would leave SM pairs without work are cut along the inner dimension: their
// ranges leave partial sums, and lora_join_kernel adds them, the adapters' term and the
// epilogue, the term in fp32 FMAs.  Most decode batches have all of their tiles there.
//
// What bounds it: the weights' bytes for few rows (1 row, K = 2560, N = 9728, R = 16: 19 us,
// 14.8 of them the bytes at the copy rate), the MMAs for many (4096 rows, R = 64: 281 us, 230 of
// them the shared product's, 20 the terms', 18 p's kernel), between them the terms of rows of several adapters, whose loads
// eight warps per SM wait for (333 rows of 37 requests, K = 1000, N = 2504: 8 of 23 us).
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

enum LoraInside { kInsideNo = 0, kInsideEach = 1, kInsideShared = 2 };   // a kernel before, each block all, the blocks together
constexpr int kInsideMost = 64;   // values of p that each block forms for itself

struct LoraMaps {
    TensorMap w[2], x;
    TensorMap b[2];          // [adapters][N][R]
    TensorMap p[2];          // p's terms, [M][sides R], boxes of 64 x 16
};

struct LoraPairParams {
    LoraParams l;
    LoraPlan plan;
    float *part;             // [rest splits][rows][256]: a range's accumulators, token by token
    int rows;                // of a tile: tn, or all that there are
    int prefetch;            // B into L2 ahead
    int inside;              // who forms p: LoraInside
    // The first stages' weights are requested before the kernel before this one is done (not where
    // that one forms p: such a call starts early as a whole): a token's call 20.3 to 18.9 us in a
    // chain, 16 rows of rank 32 27.5 to 26.5, with few tiles in ranges no change.
    int ahead;
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

// t + the products of eight bf16 values with eight fp32 ones
__device__ __forceinline__ float dot8(const uint4 &x, const float4 &y, const float4 &z, float t)
{
    t = fmaf(bf16_lo(x.x), y.x, t);
    t = fmaf(bf16_hi(x.x), y.y, t);
    t = fmaf(bf16_lo(x.y), y.z, t);
    t = fmaf(bf16_hi(x.y), y.w, t);
    t = fmaf(bf16_lo(x.z), z.x, t);
    t = fmaf(bf16_hi(x.z), z.y, t);
    t = fmaf(bf16_lo(x.w), z.z, t);
    return fmaf(bf16_hi(x.w), z.w, t);
}

// A box of a stack of matrices into this CTA's shared memory, counted on a barrier of either
// CTA of the pair.
__device__ __forceinline__ void pair_load_3d(void *dst, const TensorMap *map, int x, int y, int z, uint32_t bar)
{
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2"
        " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(smem_addr(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar)
        : "memory");
}

// The runs of 32-row blocks (the least that a pair's MMA takes as columns) with one adapter in a tile of tokens; a warp walks them.
struct LoraRuns {
    int mine, blocks, at, first, adapter;   // run: blocks first .. at - 1
    __device__ void load(const LoraParams &p, int m0, int tn)
    {
        const int lane = threadIdx.x & 31;
        blocks = min(tn / kLoraBlock, (p.M - m0 + kLoraBlock - 1) / kLoraBlock);
        mine = lane < blocks ? __ldcg(p.blocks + m0 / kLoraBlock + lane) : kNoAdapter;
        at = 0;
    }
    __device__ bool next()
    {
        while (at < blocks) {
            first = at;
            adapter = __shfl_sync(0xffffffffu, mine, at++);
            if (adapter < 0) continue;
            while (at < blocks && __shfl_sync(0xffffffffu, mine, at) == adapter) ++at;
            return true;
        }
        return false;
    }
};

// The adapters' term of 32 outputs from n0 on and 16 tokens from m0 on, a warp; mine: lanes 0
// to 15 hold the tokens' adapters, the others -1; tile(half) is called for each half of the tokens with term[token * kTermPitch + output].
constexpr int kTermPitch = 36;
constexpr int kTermWords = 8 * kTermPitch;
template <typename F>
__device__ __forceinline__ void lora_term(const LoraParams &p, int mine, int d, int sides, int64_t m0, int n0, float *term, F tile)
{
    const int lane = threadIdx.x & 31, row = lane >> 2, quad = lane & 3;
    uint32_t left = __ballot_sync(0xffffffffu, mine >= 0);
    const bool used[2] = {(left >> row & 1u) != 0, (left >> (8 + row) & 1u) != 0};
    const LoraSide &side = p.side[d];
    const float *q = p.p + (m0 + row) * sides * p.R + d * p.R + quad * 8;
    const int64_t second = 8 * static_cast<int64_t>(sides) * p.R;
    float sum[2][2][4] = {};   // halves of the tokens, halves of the outputs
    while (left) {
        // two adapters at a time, so that their rows are on the way together
        int a[2];
        uint32_t match[2];
        a[0] = __shfl_sync(0xffffffffu, mine, __ffs(left) - 1);
        match[0] = __ballot_sync(0xffffffffu, mine == a[0]);
        left &= ~match[0];
        a[1] = __shfl_sync(0xffffffffu, mine, left ? __ffs(left) - 1 : 0);
        a[1] = left ? a[1] : -1;
        match[1] = left ? __ballot_sync(0xffffffffu, mine == a[1]) : 0;
        left &= ~match[1];
        float acc[2][2][2][4] = {};
        const uint16_t *b[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) b[i] = side.b + a[i] * side.b_adapter + (n0 + row) * side.ldb + quad * 8;
        // 32 columns, two steps of the tensor cores: a lane reads 16 bytes of a row, eight columns,
        // the first four for the first step (which column sits where is free, as in the shrink)
        for (int j = 0; j < p.R; j += 32) {
            const bool in = j + quad * 8 < p.R;
            uint4 w[2][4];
            float4 v[2][2];
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    w[i][r] = in && a[i] >= 0 && n0 + row + r * 8 < p.N ? *reinterpret_cast<const uint4 *>(b[i] + r * 8 * side.ldb + j) : make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int g = 0; g < 2; ++g)
#pragma unroll
                for (int c = 0; c < 2; ++c)
                    v[g][c] = in && used[g] ? *reinterpret_cast<const float4 *>(q + g * second + j + 4 * c) : make_float4(0, 0, 0, 0);
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                uint32_t h[2][2], l[2][2];
#pragma unroll
                for (int g = 0; g < 2; ++g) {
                    const float4 x = v[g][c];
                    split_bf16x2(x.x, x.y, h[g][0], l[g][0]);
                    split_bf16x2(x.z, x.w, h[g][1], l[g][1]);
                }
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    if (a[i] < 0) continue;   // the whole warp
#pragma unroll
                    for (int t = 0; t < 2; ++t) {
                        const uint4 &x = w[i][2 * t], &y = w[i][2 * t + 1];
                        const uint32_t wa[4] = {c ? x.z : x.x, c ? y.z : y.x, c ? x.w : x.y, c ? y.w : y.y};
#pragma unroll
                        for (int g = 0; g < 2; ++g) {
                            mma_16816(acc[i][g][t], wa, h[g][0], h[g][1]);
                            mma_16816(acc[i][g][t], wa, l[g][0], l[g][1]);
                        }
                    }
                }
            }
        }
        // this lane's tokens of a half: quad * 2 and the next
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int g = 0; g < 2; ++g) {
                const bool t0 = match[i] >> (g * 8 + quad * 2) & 1u, t1 = match[i] >> (g * 8 + quad * 2 + 1) & 1u;
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    sum[g][t][0] = t0 ? acc[i][g][t][0] : sum[g][t][0];
                    sum[g][t][1] = t1 ? acc[i][g][t][1] : sum[g][t][1];
                    sum[g][t][2] = t0 ? acc[i][g][t][2] : sum[g][t][2];
                    sum[g][t][3] = t1 ? acc[i][g][t][3] : sum[g][t][3];
                }
            }
    }
#pragma unroll
    for (int g = 0; g < 2; ++g) {
        __syncwarp();
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            float *o = term + quad * 2 * kTermPitch + t * 16 + row;
            o[0] = sum[g][t][0];
            o[kTermPitch] = sum[g][t][1];
            o[8] = sum[g][t][2];
            o[kTermPitch + 8] = sum[g][t][3];
        }
        __syncwarp();
        tile(g);
    }
}

// Eight columns of p[m] from j0 on (adapter a, before its scale), summed over steps s0 .. s1 - 1
// of 256; a warp, every lane gets the sums.
__device__ __forceinline__ void lora_dot8(const LoraParams &p, int d, int64_t m, int a, int j0, int s0, int s1, float (&sum)[8])
{
    const int lane = threadIdx.x & 31;
    const LoraSide &side = p.side[d];
    const uint16_t *x = p.x + m * p.ldx, *w = side.a + a * side.a_adapter + j0 * side.lda;
#pragma unroll
    for (int i = 0; i < 8; ++i) sum[i] = 0.0f;
#pragma unroll 2
    for (int s = s0; s < s1; ++s) {
        const int k = s * 256 + lane * 8;
        const bool in = k < p.K;
        const uint4 v = in ? *reinterpret_cast<const uint4 *>(x + k) : make_uint4(0, 0, 0, 0);
        uint4 r[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) r[i] = in ? *reinterpret_cast<const uint4 *>(w + i * side.lda + k) : make_uint4(0, 0, 0, 0);
        const float4 lo = make_float4(bf16_lo(v.x), bf16_hi(v.x), bf16_lo(v.y), bf16_hi(v.y));
        const float4 hi = make_float4(bf16_lo(v.z), bf16_hi(v.z), bf16_lo(v.w), bf16_hi(v.w));
#pragma unroll
        for (int i = 0; i < 8; ++i) sum[i] = dot8(r[i], lo, hi, sum[i]);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
#pragma unroll
        for (int i = 0; i < 8; ++i) sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], o);
}

// The epilogue's eight warps (me: 0 to 7) form p: all of it at `mine`, laid out as p.p; or the
// block's share at p.p.  scratch: 2 x 8 x 8 floats.
template <int SIDES>
__device__ __forceinline__ void lora_inside(const LoraParams &p, int inside, int me, float *mine, float *scratch)
{
    const int lane = threadIdx.x & 31, per = SIDES * p.R / 8, steps = (p.K + 255) / 256;   // units of 8 columns of a row
    const int64_t units = static_cast<int64_t>(p.M) * per;
    float sum[8];
    if (inside == kInsideEach) {   // a warp per unit
        for (int64_t u = me; u < units; u += 8) {
            const int64_t m = u / per;
            const int j = static_cast<int>(u % per) * 8, a = lora_adapter(p, m);
            if (a < 0) continue;
            const int d = SIDES == 2 && j >= p.R ? 1 : 0;
            lora_dot8(p, d, m, a, j - d * p.R, 0, steps, sum);
            const float scale = p.scale ? p.scale[a] : 1.0f;
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (lane == i) mine[m * SIDES * p.R + j + i] = sum[i] * scale;
        }
        bar_sync_named(6, 256);
        return;
    }
    uint32_t turn = 0;
    for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {   // the warps share a unit's columns
        const int64_t m = u / per;
        const int j = static_cast<int>(u % per) * 8, a = lora_adapter(p, m);
        if (a < 0) continue;   // the whole block
        const int d = SIDES == 2 && j >= p.R ? 1 : 0;
        const float scale = p.scale ? p.scale[a] : 1.0f;
        lora_dot8(p, d, m, a, j - d * p.R, steps * me / 8, steps * (me + 1) / 8, sum);
        float *at = scratch + (turn++ & 1) * 64;   // written again only after the barrier behind which it was read
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (lane == i) at[me * 8 + i] = sum[i];
        bar_sync_named(6, 256);
        if (me == 0 && lane < 8) {
            float v = 0.0f;
#pragma unroll
            for (int i = 0; i < 8; ++i) v += at[i * 8 + lane];
            p.p[m * SIDES * p.R + j + lane] = v * scale;
        }
    }
}

// The same for rows that mostly have an adapter each, best of rank 16 at most (a row of more
// spreads a warp's load over 32 lines; single rows, and decode batches that the join does not
// take, come here with more): a lane has one output n, reads its row
// of each token's B, eight tokens' together, and adds the term to y.  p of 16 tokens and 16
// columns is staged in shared memory (stage, 256 floats), on the way beside B.
__device__ __forceinline__ void lora_term_rows(const LoraParams &p, int mine, const float *all_p, int d, int sides, int64_t m0, int64_t n,
                                               float *stage, float (&y)[16])
{
    const int lane = threadIdx.x & 31, R = p.R;
    const uint32_t used = __ballot_sync(0xffffffffu, mine >= 0);
    const LoraSide &side = p.side[d];
    // this lane stages 8 columns of token lane / 2
    const bool has = used >> (lane >> 1) & 1u;
    const float *q = all_p + (m0 + (lane >> 1)) * sides * R + d * R + (lane & 1) * 8;
    float4 *mystage = reinterpret_cast<float4 *>(stage + lane * 8);
    for (int j = 0; j < R; j += 16) {
        const bool in = has && j + (lane & 1) * 8 < R;
        const float4 v0 = in ? *reinterpret_cast<const float4 *>(q + j) : make_float4(0, 0, 0, 0);
        const float4 v1 = in ? *reinterpret_cast<const float4 *>(q + j + 4) : make_float4(0, 0, 0, 0);
#pragma unroll
        for (int g = 0; g < 2; ++g) {
            uint4 b[8][2];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const int a = __shfl_sync(0xffffffffu, mine, 8 * g + k);
                const uint16_t *r = side.b + a * side.b_adapter + n * side.ldb + j;
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    b[k][h] = a >= 0 && n < p.N && j + 8 * h < R ? *reinterpret_cast<const uint4 *>(r + 8 * h) : make_uint4(0, 0, 0, 0);
            }
            if (g == 0) {
                __syncwarp();
                mystage[0] = v0;
                mystage[1] = v1;
                __syncwarp();
            }
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const float4 *v = reinterpret_cast<const float4 *>(stage + (8 * g + k) * 16);
                float t = dot8(b[k][0], v[0], v[1], 0.0f);
                y[8 * g + k] += dot8(b[k][1], v[2], v[3], t);
            }
        }
    }
    __syncwarp();
}

// The exchange between the two warps of an output's g and u (as pair_tall.cuh), then the
// warps' terms.
static_assert(kPairExchange + (kInsideMost + 128) * 4 <= kPairHeader, "p and its scratch lie behind the barriers");
constexpr int kLoraSwap = 2 * 16 * 32;
constexpr uint32_t kLoraExtra = 4 * kLoraSwap * 4 + 8 * kTermWords * 4;
constexpr uint32_t kLoraSmem = kPairHeader + kPairStages * kPairStage + kLoraExtra + 1024;
static_assert(kLoraSmem <= 227 * 1024, "shared memory");

// ROWS: 16 tokens of several adapters by lora_term_rows.
template <int SIDES, bool ROWS>
__global__ void __launch_bounds__(kPairThreads, 1) lora_pair_kernel(const LoraPairParams p, const __grid_constant__ LoraMaps maps)
{
    extern __shared__ unsigned char pair_raw[];
    const PairShared s = pair_shared(pair_raw);
    const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
    const int rank = static_cast<int>(cluster_ctarank());
    const uint32_t tmem = pair_setup(s, warp);
    const LoraPlan &plan = p.plan;
    const int R = p.l.R, width = SIDES * R;
    bool ok = true;
    const int first = static_cast<int>(blockIdx.x >> 1), step = static_cast<int>(gridDim.x >> 1);
    if (!p.early && !(p.ahead && warp == 0)) {
        grid_dependency_wait();
        grid_launch_dependents();
    }
    if (p.early) grid_launch_dependents();

    if (warp == 0) {
        const uint32_t full0 = map_to_rank(s.full, 0);
        // both CTAs'; of one projection a CTA's rows are one box
        const uint32_t bytes = static_cast<uint32_t>(plan.wt) * (SIDES == 2 ? 256u : 128u) + static_cast<uint32_t>(plan.tn) * 128u;
        int st = 0, filled = 0;
        uint32_t phase = 1;
        if (p.ahead) {
            const LoraTile x = lora_tile(plan, first);
            const int n0 = x.t / plan.ttiles * plan.wt + rank * (plan.wt / 2), m0 = x.t % plan.ttiles * plan.tn + rank * (plan.tn / 2);
            filled = min(x.c1 - x.c0, kPairStages);
            for (int k = 0; k < filled; ++k) {
                unsigned char *d = s.stages + k * kPairStage;
                const uint32_t bar = full0 + static_cast<uint32_t>(k) * 8u;
                if (elect_one()) {
                    if (rank == 0) mbar_arrive_expect_tx(&s.full[k], bytes);
                    pair_load_2d(d, &maps.w[0], (x.c0 + k) * 64, n0, bar);
                    if (SIDES == 2) pair_load_2d(d + kPairOperand / 2, &maps.w[1], (x.c0 + k) * 64, n0, bar);
                }
                __syncwarp();
            }
            grid_dependency_wait();
            grid_launch_dependents();
            for (int k = 0; k < filled; ++k) {
                if (elect_one())
                    pair_load_2d(s.stages + k * kPairStage + kPairOperand, &maps.x, (x.c0 + k) * 64, m0, full0 + static_cast<uint32_t>(k) * 8u);
                __syncwarp();
            }
            st = filled % kPairStages;
            phase = filled == kPairStages ? 0 : 1;
        }
        const int done = filled;   // of the first tile
        for (int i = first; i < plan.items && ok; i += step) {
            const LoraTile x = lora_tile(plan, i);
            const int n0 = x.t / plan.ttiles * plan.wt + rank * (plan.wt / 2), m0 = x.t % plan.ttiles * plan.tn + rank * (plan.tn / 2);
            // the table: but for the first tile, whose products do not wait for it, it comes ahead
            const bool runs = p.l.blocks && x.slot < 0;
            LoraRuns run;
            if (runs && i != first) run.load(p.l, x.t % plan.ttiles * plan.tn, plan.tn);
            for (int c = x.c0 + (i == first ? done : 0); c < x.c1; ++c) {
                if (!pair_wait(&s.empty[st], phase, kWaitLimitNs)) {
                    ok = false;
                    break;
                }
                unsigned char *d = s.stages + st * kPairStage;
                const uint32_t bar = full0 + static_cast<uint32_t>(st) * 8u;
                if (elect_one()) {
                    if (rank == 0) mbar_arrive_expect_tx(&s.full[st], bytes);
                    pair_load_2d(d, &maps.w[0], c * 64, n0, bar);
                    if (SIDES == 2) pair_load_2d(d + kPairOperand / 2, &maps.w[1], c * 64, n0, bar);
                    pair_load_2d(d + kPairOperand, &maps.x, c * 64, m0, bar);
                }
                __syncwarp();
                filled += filled < kPairStages;
                if (++st == kPairStages) {
                    st = 0;
                    phase ^= 1;
                }
            }
            if (!runs || !ok) continue;
            if (i == first) {
                if (p.early) grid_dependency_wait();   // p and the table
                run.load(p.l, x.t % plan.ttiles * plan.tn, plan.tn);
            }
            while (ok && run.next()) {
                const int blocks = run.at - run.first;
                const int row = x.t % plan.ttiles * plan.tn + run.first * kLoraBlock + rank * blocks * 16;   // each CTA brings half of the run
                for (int c = 0; c < width && ok; c += 64)
                    for (int term = 0; term < 2; ++term) {
                        if (!pair_wait(&s.empty[st], phase, kWaitLimitNs)) {
                            ok = false;
                            break;
                        }
                        unsigned char *d = s.stages + st * kPairStage;
                        const uint32_t bar = full0 + static_cast<uint32_t>(st) * 8u;
                        if (elect_one()) {
                            if (rank == 0)
                                mbar_arrive_expect_tx(&s.full[st], static_cast<uint32_t>(plan.wt) * (SIDES == 2 ? 256u : 128u) + static_cast<uint32_t>(blocks) * 4096u);
                            pair_load_3d(d, &maps.b[0], c, n0, run.adapter, bar);
                            if (SIDES == 2) pair_load_3d(d + kPairOperand / 2, &maps.b[1], c - R, n0, run.adapter, bar);
                            for (int b = 0; b < blocks; ++b) pair_load_2d(d + kPairOperand + b * 2048, &maps.p[term], c, row + b * 16, bar);
                        }
                        __syncwarp();
                        filled += filled < kPairStages;
                        if (++st == kPairStages) {
                            st = 0;
                            phase ^= 1;
                        }
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
                const bool runs = p.l.blocks && x.slot < 0;
                LoraRuns run;
                if (runs && i != first) run.load(p.l, x.t % plan.ttiles * plan.tn, plan.tn);
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
                    }
                    __syncwarp();
                    if (++st == kPairStages) {
                        st = 0;
                        phase ^= 1;
                    }
                }
                if (runs && ok) {
                    if (i == first) {
                        if (p.early) grid_dependency_wait();
                        run.load(p.l, x.t % plan.ttiles * plan.tn, plan.tn);
                    }
                    while (ok && run.next()) {
                        const int cols = (run.at - run.first) * kLoraBlock;
                        const uint32_t run_idesc = tc_idesc_bf16(256, 256) - (static_cast<uint32_t>((256 - cols) >> 3) << 17);
                        const uint32_t d = tmem + buf * kPairTile + static_cast<uint32_t>(run.first * kLoraBlock);
                        for (int c = 0; c < width && ok; c += 64) {
                            const int steps = min(4, (width - c + 15) / 16);
                            for (int term = 0; term < 2; ++term) {
                                if (!pair_wait(&s.full[st], phase, kWaitLimitNs)) {
                                    ok = false;
                                    break;
                                }
                                tc_fence_after();
                                const uint64_t a = a0 + static_cast<uint32_t>(st) * (kPairStage >> 4), b = b0 + static_cast<uint32_t>(st) * (kPairStage >> 4);
                                if (elect_one()) {
                                    for (int kk = 0; kk < steps; ++kk) pair_mma_bf16(d, a + 2 * kk, b + 2 * kk, run_idesc, true);
                                    pair_commit(&s.empty[st]);
                                }
                                __syncwarp();
                                if (++st == kPairStages) {
                                    st = 0;
                                    phase ^= 1;
                                }
                            }
                        }
                    }
                }
                if (elect_one() && ok) pair_commit(&s.acc_full[buf]);
                __syncwarp();
                buf ^= 1;
                if (buf == 0) acc_phase ^= 1;
            }
        }
    } else if (warp == 2 && p.prefetch) {
        // B is read row by row at the end, where nothing hides the way, but for blocks of one
        // adapter: where it is small its bytes come into L2 beside the weights
        for (int i = first; i < plan.whole + plan.rest; i += step) {
            const LoraTile x = lora_tile(plan, i);
            const int n0 = x.t / plan.ttiles * plan.wt + rank * (plan.wt / 2), rows = min(plan.wt / 2, p.l.N - n0);
            const int m0 = x.t % plan.ttiles * plan.tn;
            for (int k = 0; k < plan.tn && m0 + k < p.l.M && rows > 0; k += 32) {
                const int m = m0 + k + lane, a = lora_adapter(p.l, m);
                const int head = __shfl_sync(0xffffffffu, a, 0), before = __shfl_up_sync(0xffffffffu, a, 1);
                if (p.l.blocks && x.slot < 0 && __all_sync(0xffffffffu, a == head || m >= p.l.M)) continue;
                if (a < 0 || (lane > 0 && a == before)) continue;
#pragma unroll
                for (int d = 0; d < SIDES; ++d) {
                    const LoraSide &side = p.l.side[d];
                    if (side.ldb == R) bulk_prefetch_l2(side.b + a * side.b_adapter + n0 * side.ldb, static_cast<uint32_t>(rows * R * 2));
                }
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
        const float *all_p = p.l.p;
        if constexpr (ROWS) {
            if (p.inside != kInsideNo) lora_inside<SIDES>(p.l, p.inside, warp - kPairEpilogue, s.exchange, s.exchange + kInsideMost);
            if (p.inside == kInsideEach) all_p = s.exchange;
        }
        uint32_t v = 0, sets = 0;
        for (int i = first; i < plan.items; i += step, ++v) {
            const LoraTile x = lora_tile(plan, i);
            const uint32_t buf = v & 1;
            const int n0 = x.t / plan.ttiles * plan.wt + rank * (plan.wt / 2) + row0;
            const int n = row0 + lane < plan.wt / 2 ? n0 + lane : p.l.N;   // N: none
            const int m0 = x.t % plan.ttiles * plan.tn + half * (plan.tn / 2);
            // the tokens' adapters, a lane per token, on the way while the products run
            int ids[4];
#pragma unroll
            for (int b = 0; b < 4; ++b) ids[b] = p.l.adapters > 0 && b * 32 < plan.tn / 2 ? lora_adapter(p.l, static_cast<int64_t>(m0) + b * 32 + lane) : -1;
            // and the table's entries of this half of the tile
            const int entry = p.l.blocks && x.slot < 0 && lane < 5 && m0 / kLoraBlock + lane <= (p.l.M - 1) / kLoraBlock
                                  ? __ldcg(p.l.blocks + m0 / kLoraBlock + lane) : kNoAdapter;
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
                    float *o = p.part + (static_cast<int64_t>(x.slot) * p.rows + half * (plan.tn / 2) + j) * 256 + rank * 128 + q * 32 + lane;
#pragma unroll
                    for (int k = 0; k < 16; ++k)
                        if (k < tokens) __stcg(o + k * 256, __uint_as_float(r[k]));
                    continue;   // the whole tile, in every warp: no exchange is begun
                }
                float y[16];
#pragma unroll
                for (int k = 0; k < 16; ++k) y[k] = __uint_as_float(r[k]);
                const int at32 = j >> 5, id = at32 == 0 ? ids[0] : at32 == 1 ? ids[1] : at32 == 2 ? ids[2] : ids[3];
                int mine = __shfl_sync(0xffffffffu, id, (j & 16) + (lane & 15));   // these 16 tokens', in the first lanes
                if (lane >= 16) mine = -1;
                const int block = __shfl_sync(0xffffffffu, entry, (m0 + j) / kLoraBlock - m0 / kLoraBlock);
                const bool term_here = p.inside == kInsideEach || block == kMixed;
                if (tokens > 0 && term_here) {
                    if constexpr (ROWS)
                        lora_term_rows(p.l, mine, all_p, d, SIDES, static_cast<int64_t>(m0) + j, n, term, y);
                    else
                        lora_term(p.l, mine, d, SIDES, static_cast<int64_t>(m0) + j, n0, term, [&](int g) {
#pragma unroll
                            for (int k = 0; k < 16; ++k)
                                if (k >> 3 == g) y[k] += term[(k & 7) * kTermPitch + lane];
                        });
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
// warp takes 32 outputs and TOKENS tokens.  LANES lanes share a row of B, eight columns each (R
// <= 8 LANES), so that a load of the warp is 512 consecutive bytes; LANES - 1 shuffles leave each
// output's sum in one lane.  Here an SM has 24 to 64 warps, beside the products it has eight
// for this: 48 rows with adapters of rank 64 of their own took 83 us there, 57 here.
template <int SIDES, int TOKENS, int LANES>
__global__ void __launch_bounds__(256) lora_join_kernel(const LoraPairParams p)
{
    constexpr int kRows = 32 / LANES;                 // rows of a load
    const LoraPlan &plan = p.plan;
    const int lane = threadIdx.x & 31, part = lane % LANES, row = lane / LANES, R = p.l.R;
    const int from = lane % kRows * LANES + lane / kRows;   // where the sum of output `lane` ends up
    const int groups = plan.tn / TOKENS, blocks = (plan.wt + 31) / 32;   // of a tile
    const int64_t total = static_cast<int64_t>(plan.rest) * blocks * groups;
    grid_dependency_wait();
    grid_launch_dependents();
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5); i < total; i += static_cast<int64_t>(gridDim.x) * 8) {
        // tiles' first tokens first: those behind the last row cost nothing
        const int group = static_cast<int>(i / (plan.rest * blocks)), other = static_cast<int>(i % (plan.rest * blocks));
        const int tile = other / blocks, j0 = group * TOKENS, w = other % blocks * 32;
        const int t = plan.whole + tile, n0 = t / plan.ttiles * plan.wt + w;
        const int64_t m0 = static_cast<int64_t>(t % plan.ttiles) * plan.tn + j0;
        if (m0 >= p.l.M || n0 >= p.l.N) continue;   // the whole warp
        const bool mine = w + lane < plan.wt && n0 + lane < p.l.N;
        int a[TOKENS];
#pragma unroll
        for (int k = 0; k < TOKENS; ++k) a[k] = lora_adapter(p.l, m0 + k);
        // output w of the tile: a CTA holds wt / 2 of them, in dual tiles from lanes 0 and 64 on
        const int rank = w + lane >= plan.wt / 2 ? 1 : 0, at = rank * 128 + w + lane - rank * (plan.wt / 2);
        float acc[TOKENS][SIDES] = {};
        const float *q = p.part + (static_cast<int64_t>(tile) * p.rows + j0) * 256 + at;
#pragma unroll 4
        for (int s = 0; s < plan.splits; ++s, q += static_cast<int64_t>(plan.rest) * p.rows * 256)
#pragma unroll
            for (int k = 0; k < TOKENS; ++k)
#pragma unroll
                for (int d = 0; d < SIDES; ++d) acc[k][d] += mine && m0 + k < p.l.M ? __ldcg(q + k * 256 + d * 64) : 0.0f;
#pragma unroll
        for (int d = 0; d < SIDES; ++d) {
            const LoraSide &side = p.l.side[d];
            uint4 b[TOKENS][LANES];
            float4 v[TOKENS][2];
#pragma unroll
            for (int k = 0; k < TOKENS; ++k) {
                const uint16_t *r = side.b + a[k] * side.b_adapter + (n0 + row) * static_cast<int64_t>(side.ldb) + part * 8;
                const float *x = p.l.p + (m0 + k) * SIDES * R + d * R + part * 8;
                const bool has = a[k] >= 0 && part * 8 < R;
#pragma unroll
                for (int h = 0; h < LANES; ++h)
                    b[k][h] = has && n0 + h * kRows + row < p.l.N ? *reinterpret_cast<const uint4 *>(r + h * kRows * side.ldb) : make_uint4(0, 0, 0, 0);
                v[k][0] = has ? *reinterpret_cast<const float4 *>(x) : make_float4(0, 0, 0, 0);
                v[k][1] = has ? *reinterpret_cast<const float4 *>(x + 4) : make_float4(0, 0, 0, 0);
            }
#pragma unroll
            for (int k = 0; k < TOKENS; ++k) {
                float sum[LANES];
#pragma unroll
                for (int h = 0; h < LANES; ++h) sum[h] = dot8(b[k][h], v[k][0], v[k][1], 0.0f);
                // halves are exchanged until a lane has one sum: of the rows' group `part`
#pragma unroll
                for (int o = LANES / 2; o > 0; o >>= 1) {
                    const bool upper = part & o;
#pragma unroll
                    for (int h = 0; h < o; ++h) {
                        const float theirs = __shfl_xor_sync(0xffffffffu, upper ? sum[h] : sum[h + o], o);
                        sum[h] = (upper ? sum[h + o] : sum[h]) + theirs;
                    }
                }
                acc[k][d] += __shfl_sync(0xffffffffu, sum[0], from);
            }
        }
        __syncwarp();
        if (!mine) continue;
#pragma unroll
        for (int k = 0; k < TOKENS; ++k) {
            if (m0 + k >= p.l.M) break;
            uint16_t *o = p.l.out + (m0 + k) * p.l.ldo + n0 + lane;
            const float g = acc[k][0], u = acc[k][SIDES - 1];
            if constexpr (SIDES == 2)
                *o = p.l.mode == 0 ? f32_to_bf16(silu_short(g) * u) : static_cast<uint16_t>(glu_hf_short(g, u));
            else
                *o = f32_to_bf16(g);
        }
    }
}

}  // namespace mbglu
