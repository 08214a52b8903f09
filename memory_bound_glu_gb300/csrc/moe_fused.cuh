// moe_fused.cuh -- the expert layer of a decode batch in one cooperative kernel: one
// block per SM, all resident at once, that meet at three to five grid barriers.
//
//   1  logits, a warp per expert and four tokens                        | barrier
//   2  the choice, by every block for itself, or of many tokens by a block each   (| barrier)
//   3  gated projections of the chosen experts                          | barrier
//   4  activation, as two bf16 terms                                    (| barrier, unless 3 does it)
//   5  down projections                                                 | barrier
//   6  weighted sum over a token's experts
//
// What bounds it are the chosen experts' weights.  In 3 and 5 they are the MMA's 128-row
// side (tcgen05, accumulators in tensor memory): a unit is a 16 KB box of 64 columns,
// of 64 gate and 64 up rows or of 128 down rows.  The units of all tiles of all chosen
// experts form one sequence that is cut into equal ranges, one per block, so every SM
// reads the same number of bytes whatever was chosen; a tile that a border cuts leaves
// parts of its sum, which whoever needs the sum adds in the order of the blocks.  Where the
// tiles are fewer than the blocks and at least half as many -- half of the SMs still draw the
// memory's full rate -- a block has one whole tile, and 4 is done where 3's sums are read, with
// no barrier between (a token of 8 x 12 tiles: 29.7 to 28.5 us).  The
// side of the tokens: in 3 all tokens for every expert (a column costs nothing beside the
// weights; only the chosen ones are written), in 5 the activation rows of the expert.
// A token's column is its own, so what other tokens hold does not reach it.
//
// In 5 the activation's second terms are more rows of the tokens' side, so their products
// are more columns of the same MMA (added up where they are read) and the weights are read
// from shared memory once: as MMAs of their own they took a unit from 0.2 to 0.3 us.
//
// The copies of weights run ahead over the barriers: the first units of 5 are on their
// way while 3 is finished and 4 runs, up to the ring's 96 to 160 KB per SM.
//
// Roles (384 threads): warp 0 copies weights, warp 2 the tokens' side, warp 1 owns the
// tensor memory and issues the MMAs, warps 4-7 read accumulators, warps 4-11 do 4 and 6,
// all warps 1 and 2.  Every wait is bounded; after one gives up, or finds a counter that was not 0
// at the start, each role ends without touching memory, and the counters are marked.
#pragma once
#include "dense_common.cuh"
#include "moe_route.cuh"
#include "stack_copy.cuh"
#include "tc_pair.cuh"
#include "two_terms.cuh"

namespace mbglu {

constexpr int kMoeThreads = 384;
constexpr int kMoeWarps = kMoeThreads / 32;
constexpr int kMoeSum = 4;                        // the first warp of those that read accumulators and add
constexpr int kMoeMaxStages = 10;
constexpr uint32_t kMoeUnit = 16384;              // a unit's weights
constexpr uint32_t kMoeAcc = 128;                 // columns of an accumulator: 64 tokens' two terms
constexpr uint32_t kMoeCols = 2 * kMoeAcc;
constexpr int kMoeKeys = kMoeMaxExperts;          // logits that a block orders at a time
constexpr int kMoeSlots = kMoeMaxRows * kMoeMaxTopK;

struct MoeMaps {
    TensorMap gate, up;   // [E][N][K], boxes of 64 x 64 (columns x rows)
    TensorMap down;       // [E][K][N], 64 x 128
    TensorMap h;          // [T][K], 64 x padded tokens
    TensorMap act;        // [2 act_rows][N], 64 x 16
};

struct MoeParams {
    const uint16_t *h, *router;
    int64_t ldh, ldr, ldo;
    uint16_t *out;
    int32_t *ids;            // or null
    float *weights;          // or null
    uint32_t *counters;      // five barriers and the exit (the fifth), all 0 at the start and at the end
    int32_t *chosen;         // [T][top_k]: what the blocks choose, where each has tokens of its own
    float *chosen_weight;
    float *logits;           // [T][E]
    float *gu;               // [slots][2 N]: g, then u
    float *y;                // [slots][K]
    float *carry;            // [blocks][pad][128]: the part of a block's first tile that began in an earlier block
    uint16_t *act;           // [2 act_rows][act_ld]: first terms, then second ones
    int64_t act_ld;
    int act_rows;
    int T, E, top_k, N, K, renormalize;
    int pad;                 // tokens padded to a multiple of 16
    int stages;
};

struct alignas(16) MoeShared {
    uint64_t weights_full[kMoeMaxStages], tokens_full[kMoeMaxStages], empty[kMoeMaxStages];
    uint64_t acc_full[2], acc_empty[2], act_ready, done;
    uint32_t tmem, failed;                       // failed: any thread sets it at any time
    // The same for those that meet at named barriers and have to leave together: written only in
    // front of the barrier behind which they read it.
    uint32_t phase_failed, tile_failed;
    int active, pad_;
    uint64_t mask[kMoeMaxExperts];               // tokens that chose the expert (little-endian halves are set)
    alignas(16) uint32_t key[kMoeKeys];          // the logits that the block orders
    float2 pairs[kMoeWarps][4];                  // logits' parts
    int chunk_used[kMoeMaxExperts / 32], chunk_slots[kMoeMaxExperts / 32];
    float weight[kMoeSlots];
    uint16_t id[kMoeSlots];                      // [T][top_k]
    uint16_t expert[kMoeMaxExperts], first[kMoeMaxExperts + 1];   // of the i-th chosen expert: itself, its first slot
    uint16_t where[kMoeMaxExperts];              // an expert's place among the chosen ones
    uint16_t of_slot[kMoeSlots];                 // a slot's place among the chosen experts
    float4 sums[kMoeWarps - kMoeSum][32];        // 6: what the warps of a team add up
};

constexpr uint32_t kMoeHeader = (sizeof(MoeShared) + 1023) / 1024 * 1024;
__host__ __device__ constexpr uint32_t moe_stage_bytes(int pad) { return kMoeUnit + 256u * static_cast<uint32_t>(pad); }
constexpr uint32_t kMoeSmemMost = 227 * 1024;     // no number of tokens takes more
__host__ __device__ constexpr int moe_stages(int pad)
{
    const int n = static_cast<int>((kMoeSmemMost - kMoeHeader - 1024) / moe_stage_bytes(pad));
    return n < kMoeMaxStages ? n : kMoeMaxStages;
}
__host__ __device__ constexpr uint32_t moe_smem(int pad) { return kMoeHeader + 1024 + static_cast<uint32_t>(moe_stages(pad)) * moe_stage_bytes(pad); }

// Orders this thread's plain accesses to any memory against asynchronous copies'.
__device__ __forceinline__ void fence_proxy_async_all() { asm volatile("fence.proxy.async;" ::: "memory"); }

__device__ __forceinline__ uint32_t ld_acquire_gpu(const uint32_t *p)
{
    uint32_t v;
    asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
    return v;
}

__device__ __forceinline__ uint32_t add_acq_rel_gpu(uint32_t *p, uint32_t v)
{
    uint32_t old;
    asm volatile("atom.add.acq_rel.gpu.global.u32 %0, [%1], %2;" : "=r"(old) : "l"(p), "r"(v) : "memory");
    return old;
}

// One thread per block, after a barrier of the threads whose writes it publishes; and before
// one of those that read what the other blocks published.  A counter that goes beyond the blocks
// did not begin at 0 (an earlier call gave up, or another use of the workspace wrote there): false.
__device__ __forceinline__ void grid_arrive(uint32_t *counter)
{
    asm volatile("red.release.gpu.global.add.u32 [%0], 1;" ::"l"(counter) : "memory");
}
__device__ __forceinline__ bool grid_wait(const uint32_t *counter, uint64_t limit_ns)
{
    uint64_t t0 = 0;
    for (uint32_t i = 1;; ++i) {
        const uint32_t v = ld_acquire_gpu(counter);
        if (v >= gridDim.x) return v == gridDim.x;
        if ((i & 63u) == 0) {
            const uint64_t now = global_timer_ns();
            if (t0 == 0)
                t0 = now;
            else if (now - t0 > limit_ns)
                return false;
        }
    }
}

// A block that fails marks every counter: the other blocks' barriers end at once, and so does any
// later call on the workspace, until its counters are zeroed.
constexpr int kMoeCounters = 6;
__device__ __forceinline__ void grid_fail(uint32_t *counters)
{
    for (int i = 0; i < kMoeCounters; ++i) atomicOr(counters + i, 0x80000000u);
}

// The units of a phase: `chosen` experts x `tiles` x `chunks`, cut into ranges for the
// first `blocks` blocks.
struct MoeUnits {
    uint32_t tiles, chunks, total, blocks;
    bool whole;              // one tile per block
};

__device__ __forceinline__ MoeUnits moe_units(int chosen, int tiles, int chunks)
{
    MoeUnits u;
    u.tiles = static_cast<uint32_t>(tiles);
    u.chunks = static_cast<uint32_t>(chunks);
    u.total = static_cast<uint32_t>(chosen) * u.tiles * u.chunks;
    const uint32_t all = static_cast<uint32_t>(chosen) * u.tiles;
    u.whole = all <= gridDim.x && 2 * all >= gridDim.x;
    u.blocks = u.whole ? all : min(gridDim.x, u.total);
    return u;
}
// block b's first unit; total * blocks fits 32 bits
__device__ __forceinline__ uint32_t moe_begin(const MoeUnits &u, uint32_t b) { return b >= u.blocks ? u.total : u.total * b / u.blocks; }
__device__ __forceinline__ uint32_t moe_owner(const MoeUnits &u, uint32_t unit) { return ((unit + 1) * u.blocks - 1) / u.total; }

// A walk over a block's units.
struct MoeWalk {
    uint32_t left, chunk, tile, expert;   // expert: its place among the chosen ones
    __device__ MoeWalk(const MoeUnits &u)
    {
        const uint32_t at = moe_begin(u, blockIdx.x);
        left = moe_begin(u, blockIdx.x + 1) - at;
        const uint32_t q = at / u.chunks;
        chunk = at - q * u.chunks;
        expert = q / u.tiles;
        tile = q - expert * u.tiles;
    }
    __device__ void next(const MoeUnits &u)
    {
        --left;
        if (++chunk == u.chunks) next_tile(u);
    }
    __device__ void next_tile(const MoeUnits &u)
    {
        chunk = 0;
        if (++tile == u.tiles) {
            tile = 0;
            ++expert;
        }
    }
    // units of this tile in the block's range
    __device__ uint32_t run(const MoeUnits &u) const { return min(left, u.chunks - chunk); }
};

// Up to four tokens' logits of one expert (one token: four chains of one), as sums (s, c) over
// every parts-th 256 columns from the part-th on; a warp.  The next columns are on the way
// while these are summed.
template <int TOKENS>
__device__ __forceinline__ void moe_logits(const MoeParams &p, int e, int t0, int part, int parts, float (&s)[4], float (&c)[4])
{
    const int lane = threadIdx.x & 31;
    const uint16_t *w = p.router + e * p.ldr, *h = p.h + t0 * p.ldh;
    uint4 b, a[TOKENS];
    const auto load = [&](int k) {
        const bool in = k < p.K;
        b = in ? *reinterpret_cast<const uint4 *>(w + k) : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int j = 0; j < TOKENS; ++j) a[j] = in && t0 + j < p.T ? *reinterpret_cast<const uint4 *>(h + j * p.ldh + k) : make_uint4(0, 0, 0, 0);
    };
#pragma unroll
    for (int j = 0; j < 4; ++j) s[j] = c[j] = 0.0f;
    int k = part * 256 + lane * 8;
    load(k);
    for (int k0 = part * 256; k0 < p.K; k0 += parts * 256) {
        const uint32_t bw[4] = {b.x, b.y, b.z, b.w};
        uint32_t aw[TOKENS][4];
#pragma unroll
        for (int j = 0; j < TOKENS; ++j) {
            aw[j][0] = a[j].x;
            aw[j][1] = a[j].y;
            aw[j][2] = a[j].z;
            aw[j][3] = a[j].w;
        }
        k += parts * 256;
        load(k);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < TOKENS; ++j) {
                const int at = TOKENS > 1 ? j : i;
                two_sum(s[at], c[at], __fmul_rn(bf16_lo(aw[j][i]), bf16_lo(bw[i])));
                two_sum(s[at], c[at], __fmul_rn(bf16_hi(aw[j][i]), bf16_hi(bw[i])));
            }
    }
    if (TOKENS == 1) {
#pragma unroll
        for (int i = 1; i < 4; ++i) two_sum(s[0], c[0], s[i], c[i]);
    }
#pragma unroll
    for (int j = 0; j < TOKENS; ++j) warp_pair_sum(s[j], c[j]);
}

// The logits of all tokens, over all blocks.  Where there are fewer pairs of an expert and
// four tokens than warps, several warps share a pair's columns.
template <int TOKENS>
__device__ __forceinline__ void moe_all_logits(const MoeParams &p, MoeShared &sh, int warp)
{
    const int lane = threadIdx.x & 31, groups = (p.T + TOKENS - 1) / TOKENS, items = p.E * groups, grid = static_cast<int>(gridDim.x);
    int parts = 1;   // a divisor of the warps
    if (items <= grid)
        parts = 12;
    else if (items <= 2 * grid)
        parts = 6;
    else if (items <= 3 * grid)
        parts = 4;
    else if (items <= 6 * grid)
        parts = 2;
    static_assert(kMoeWarps == 12, "parts");
    const int part = warp % parts;
    for (int i = warp / parts * grid + static_cast<int>(blockIdx.x); i < items; i += kMoeWarps / parts * grid) {
        const int e = i / groups, t0 = i % groups * TOKENS;
        float s[4], c[4];
        moe_logits<TOKENS>(p, e, t0, part, parts, s, c);
        if (lane == 0) {
#pragma unroll
            for (int j = 0; j < TOKENS; ++j) {
                if (parts > 1)
                    sh.pairs[warp][j] = make_float2(s[j], c[j]);
                else if (t0 + j < p.T)
                    __stcg(p.logits + (t0 + j) * p.E + e, pair_value(s[j], c[j]));
            }
        }
    }
    if (parts == 1) return;   // the whole block
    __syncthreads();          // with several parts there is one round of pairs
    const int i = warp / parts * grid + static_cast<int>(blockIdx.x);
    if (part == 0 && i < items && lane < TOKENS) {
        const int e = i / groups, t = i % groups * TOKENS + lane;
        float2 v = sh.pairs[warp][lane];
        for (int w = 1; w < parts; ++w) two_sum(v.x, v.y, sh.pairs[warp + w][lane].x, sh.pairs[warp + w][lane].y);
        if (t < p.T) __stcg(p.logits + t * p.E + e, pair_value(v.x, v.y));
    }
}

// The choice of `tokens` tokens from t0 on, by the block.  A thread has an expert and counts
// those before it (larger, or equal with a lower index): its place.  No step waits for
// another, which a search for one maximum after the other does (8 of 128 by shuffles took
// 4 us where this takes 1).
__device__ __forceinline__ void moe_order(const MoeParams &p, MoeShared &s, int t0, int tokens)
{
    const int pitch = (p.E + 3) & ~3, total = tokens * pitch;
    for (int i = threadIdx.x; i < total; i += kMoeThreads) {
        const int t = i / pitch, e = i - t * pitch;
        s.key[i] = e < p.E ? order_key(__ldcg(p.logits + (t0 + t) * p.E + e)) : 0u;   // 0: no expert
    }
    __syncthreads();
    for (int i = threadIdx.x; i < total; i += kMoeThreads) {
        const int t = i / pitch, e = i - t * pitch;
        const uint32_t mine = s.key[i];
        const uint4 *k = reinterpret_cast<const uint4 *>(s.key + t * pitch);
        int place = 0;
#pragma unroll 4
        for (int q = 0; q < pitch / 4; ++q) {
            const uint4 v = k[q];   // no key is the largest number
            place += (v.x + (4 * q < e) > mine) + (v.y + (4 * q + 1 < e) > mine) + (v.z + (4 * q + 2 < e) > mine) + (v.w + (4 * q + 3 < e) > mine);
        }
        if (mine != 0 && place < p.top_k) s.id[(t0 + t) * p.top_k + place] = static_cast<uint16_t>(e);
    }
    __syncthreads();
}

// The weights of what moe_order has chosen; a warp per token, `warps` of them.
__device__ __forceinline__ void moe_weigh(const MoeParams &p, MoeShared &s, int t0, int tokens, int warp, int warps)
{
    const int lane = threadIdx.x & 31, pitch = (p.E + 3) & ~3;
    for (int t = warp; t < tokens; t += warps) {
        const uint16_t *id = s.id + (t0 + t) * p.top_k;
        const uint32_t *k = s.key + t * pitch;
        const float top = key_value(k[id[0]]);
        const float e = lane < p.top_k ? expf(key_value(k[id[lane < p.top_k ? lane : 0]]) - top) : 0.0f;
        float sum = p.renormalize ? e : 0.0f;
        bool nan = false;
        for (int i = lane; i < p.E; i += 32) {
            nan = nan || k[i] == 1;
            if (!p.renormalize) sum += expf(key_value(k[i]) - top);
        }
        nan = __any_sync(0xffffffffu, nan);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        if (lane < p.top_k) s.weight[(t0 + t) * p.top_k + lane] = nan ? __uint_as_float(0x7fffffffu) : e / sum;
    }
}

// Whether each block chooses for all tokens.
__device__ __forceinline__ bool moe_choose_all(const MoeParams &p) { return p.T * ((p.E + 3) & ~3) <= kMoeKeys; }

// 2: the choice of all tokens, and from it the tables of the chosen experts; false after a
// wait that gave up, in every thread.
__device__ __forceinline__ bool moe_choose(const MoeParams &p, MoeShared &s, int warp)
{
    const int lane = threadIdx.x & 31, slots = p.T * p.top_k;
    if (moe_choose_all(p)) {
        moe_order(p, s, 0, p.T);   // the weights are for 6 and come while the copies run
        if (blockIdx.x == 0 && p.ids)
            for (int i = threadIdx.x; i < slots; i += kMoeThreads) p.ids[i] = s.id[i];
    } else {
        for (int t = static_cast<int>(blockIdx.x); t < p.T; t += static_cast<int>(gridDim.x)) {
            moe_order(p, s, t, 1);
            if (warp == 0) {
                moe_weigh(p, s, t, 1, 0, 1);
                __syncwarp();
                if (lane < p.top_k) {
                    const int i = t * p.top_k + lane;
                    __stcg(p.chosen + i, static_cast<int32_t>(s.id[i]));
                    __stcg(p.chosen_weight + i, s.weight[i]);
                    if (p.ids) p.ids[i] = s.id[i];
                    if (p.weights) p.weights[i] = s.weight[i];
                }
            }
            __syncthreads();
        }
        __syncthreads();
        if (threadIdx.x == 0) {
            grid_arrive(p.counters + 5);
            if (!grid_wait(p.counters + 5, kWaitLimitNs)) s.failed = 1;
        }
        __syncthreads();
        if (s.failed != 0) return false;
        for (int i = threadIdx.x; i < slots; i += kMoeThreads) {
            // behind a barrier that did not hold anything may lie there: an index of the tables all the same
            s.id[i] = static_cast<uint16_t>(min(static_cast<uint32_t>(__ldcg(p.chosen + i)), static_cast<uint32_t>(p.E - 1)));
            s.weight[i] = __ldcg(p.chosen_weight + i);
        }
        __syncthreads();
    }
    if (p.T == 1) {   // the choice is the table, in its own order
        if (static_cast<int>(threadIdx.x) < p.top_k) {
            const int i = static_cast<int>(threadIdx.x), e = s.id[i];
            s.mask[e] = 1;
            s.expert[i] = static_cast<uint16_t>(e);
            s.where[e] = s.first[i] = s.of_slot[i] = static_cast<uint16_t>(i);
            if (i == 0) {
                s.active = p.top_k;
                s.first[p.top_k] = static_cast<uint16_t>(p.top_k);
            }
        }
        __syncthreads();
        return true;
    }
    for (int i = threadIdx.x; i < slots; i += kMoeThreads)
        atomicOr(reinterpret_cast<uint32_t *>(&s.mask[s.id[i]]) + (i / p.top_k >> 5), 1u << (i / p.top_k & 31));
    __syncthreads();
    // 32 experts at a time: how many are used, by how many tokens
    const int chunks = (p.E + 31) / 32;
    for (int i = warp; i < chunks; i += kMoeWarps) {
        const int e = i * 32 + lane, count = e < p.E ? __popcll(s.mask[e]) : 0;
        const uint32_t used = __ballot_sync(0xffffffffu, count > 0);
        const int total = __reduce_add_sync(0xffffffffu, count);
        if (lane == 0) {
            s.chunk_used[i] = __popc(used);
            s.chunk_slots[i] = total;
        }
    }
    __syncthreads();
    for (int i = warp; i < chunks; i += kMoeWarps) {
        const int e = i * 32 + lane, count = e < p.E ? __popcll(s.mask[e]) : 0;
        const uint32_t used = __ballot_sync(0xffffffffu, count > 0);
        // the chunks before this one
        const int n = __reduce_add_sync(0xffffffffu, lane < i ? s.chunk_used[lane] : 0);
        const int base = __reduce_add_sync(0xffffffffu, lane < i ? s.chunk_slots[lane] : 0);
        int before = count;   // inclusive sum over the lanes
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, before, o);
            if (lane >= o) before += v;
        }
        const int at = n + __popc(used & ((1u << lane) - 1)), first = base + before - count;
        if (count > 0) {
            s.expert[at] = static_cast<uint16_t>(e);
            s.first[at] = static_cast<uint16_t>(first);
            s.where[e] = static_cast<uint16_t>(at);
            for (int j = 0; j < count; ++j) s.of_slot[first + j] = static_cast<uint16_t>(at);
        }
        if (i == chunks - 1 && lane == 31) {
            s.active = n + __popc(used);
            s.first[n + __popc(used)] = static_cast<uint16_t>(base + before);
        }
    }
    __syncthreads();
    return true;
}

// The activation as two bf16 terms, so that the tensor cores' operand is off by 2^-18 and not
// by 2^-9.
__device__ __forceinline__ void moe_act(float g, float u, uint16_t &hi, uint16_t &lo)
{
    uint32_t h, l;
    split_bf16x2(silu_f32(g) * u, 0.0f, h, l);
    hi = static_cast<uint16_t>(h);
    lo = static_cast<uint16_t>(l);
}

// A warp, before its part of 5: the activation is there, in every lane alike; false after a failure.
// As long as the barriers of 3 and 4 take at most.
__device__ __forceinline__ bool moe_act_ready(MoeShared &s)
{
    const bool there = pair_wait(&s.act_ready, 0, 4 * kWaitLimitNs);
    return __all_sync(0xffffffffu, there && *reinterpret_cast<volatile uint32_t *>(&s.failed) == 0);
}

static __global__ void __launch_bounds__(kMoeThreads, 1) moe_fused_kernel(const MoeParams p, const __grid_constant__ MoeMaps maps)
{
    extern __shared__ unsigned char moe_raw[];
    unsigned char *base = moe_raw + ((1024u - (smem_addr(moe_raw) & 1023u)) & 1023u);
    MoeShared &s = *reinterpret_cast<MoeShared *>(base);
    unsigned char *ring = base + kMoeHeader;
    const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
    const uint32_t stage_bytes = moe_stage_bytes(p.pad);

    if (threadIdx.x == 0) {
        // the descriptors are on their way before the first copies want them
        prefetch_tensor_map(&maps.gate);
        prefetch_tensor_map(&maps.up);
        prefetch_tensor_map(&maps.down);
        prefetch_tensor_map(&maps.h);
        prefetch_tensor_map(&maps.act);
        for (int i = 0; i < p.stages; ++i) {
            mbar_init(&s.weights_full[i], 1);
            mbar_init(&s.tokens_full[i], 1);
            mbar_init(&s.empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s.acc_full[i], 1);
            mbar_init(&s.acc_empty[i], 4);
        }
        mbar_init(&s.act_ready, 1);
        mbar_init(&s.done, 1);
        s.failed = s.phase_failed = s.tile_failed = 0;
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc(&s.tmem, kMoeCols);
        tmem_relinquish();
    }
    for (int e = threadIdx.x; e < p.E; e += kMoeThreads) s.mask[e] = 0;

    // 1: logits
    if (p.T == 1)
        moe_all_logits<1>(p, s, warp);
    else
        moe_all_logits<4>(p, s, warp);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = s.tmem;
    if (threadIdx.x == 0) {
        grid_arrive(p.counters);
        if (!grid_wait(p.counters, kWaitLimitNs)) s.failed = 1;
    }
    __syncthreads();
    bool ok = s.failed == 0;

    if (ok) ok = moe_choose(p, s, warp);
    const MoeUnits gated = moe_units(ok ? s.active : 0, (p.N + 63) / 64, (p.K + 63) / 64);
    const MoeUnits down = moe_units(ok ? s.active : 0, (p.K + 127) / 128, (p.N + 63) / 64);

    if (!ok) {
        // nothing was chosen: no role has anything to do
    } else if (warp == 0) {
        const uint64_t policy = l2_policy_evict_first();
        int st = 0, issued = 0;
        uint32_t phase = 1;
        for (int second = 0; second < 2 && ok; ++second) {
            const MoeUnits &units = second ? down : gated;
            for (MoeWalk w(units); w.left > 0; w.next(units)) {
                if (!pair_wait(&s.empty[st], phase, kWaitLimitNs)) {
                    ok = false;
                    break;
                }
                if (elect_one()) {
                    unsigned char *d = ring + st * stage_bytes;
                    const int e = s.expert[w.expert], x = static_cast<int>(w.chunk) * 64;
                    mbar_arrive_expect_tx(&s.weights_full[st], kMoeUnit);
                    if (!second) {
                        tma_load_3d(d, &maps.gate, x, static_cast<int>(w.tile) * 64, e, &s.weights_full[st], policy);
                        tma_load_3d(d + kMoeUnit / 2, &maps.up, x, static_cast<int>(w.tile) * 64, e, &s.weights_full[st], policy);
                    } else {
                        tma_load_3d(d, &maps.down, x, static_cast<int>(w.tile) * 128, e, &s.weights_full[st], policy);
                    }
                }
                __syncwarp();
                issued += issued < p.stages;
                if (++st == p.stages) {
                    st = 0;
                    phase ^= 1;
                }
            }
        }
        // no copy may be in flight when the block leaves
        for (int i = 0; i < issued; ++i) {
            int at = st - issued + i;
            const uint32_t ph = at < 0 ? phase : phase ^ 1;
            if (at < 0) at += p.stages;
            if (!pair_wait(&s.weights_full[at], ph, kWaitLimitNs)) ok = false;
        }
    } else if (warp == 2) {
        const uint64_t policy = l2_policy_evict_last();
        int st = 0, issued = 0;
        uint32_t phase = 1;
        for (int second = 0; second < 2 && ok; ++second) {
            const MoeUnits &units = second ? down : gated;
            if (second) {
                ok = moe_act_ready(s);
                fence_proxy_async_all();
                if (!ok) break;
            }
            for (MoeWalk w(units); w.left > 0; w.next(units)) {
                if (!pair_wait(&s.empty[st], phase, kWaitLimitNs)) {
                    ok = false;
                    break;
                }
                if (elect_one()) {
                    unsigned char *d = ring + st * stage_bytes + kMoeUnit;
                    const int x = static_cast<int>(w.chunk) * 64;
                    if (!second) {
                        mbar_arrive_expect_tx(&s.tokens_full[st], static_cast<uint32_t>(p.pad) * 128u);
                        tma_load_2d(d, &maps.h, x, 0, &s.tokens_full[st], policy);
                    } else {
                        const int first = s.first[w.expert], boxes = (s.first[w.expert + 1] - first + 15) / 16;
                        mbar_arrive_expect_tx(&s.tokens_full[st], static_cast<uint32_t>(boxes) * 4096u);
                        for (int i = 0; i < boxes; ++i) {
                            tma_load_2d(d + i * 2048, &maps.act, x, first + i * 16, &s.tokens_full[st], policy);
                            tma_load_2d(d + (boxes + i) * 2048, &maps.act, x, p.act_rows + first + i * 16, &s.tokens_full[st], policy);
                        }
                    }
                }
                __syncwarp();
                issued += issued < p.stages;
                if (++st == p.stages) {
                    st = 0;
                    phase ^= 1;
                }
            }
        }
        for (int i = 0; i < issued; ++i) {
            int at = st - issued + i;
            const uint32_t ph = at < 0 ? phase : phase ^ 1;
            if (at < 0) at += p.stages;
            if (!pair_wait(&s.tokens_full[at], ph, kWaitLimitNs)) ok = false;
        }
    } else if (warp == 1) {
        int st = 0;
        uint32_t phase = 0, buf = 0, acc_phase = 1;
        const uint64_t a0 = smem_desc_sw128(ring);
        for (int second = 0; second < 2 && ok; ++second) {
            const MoeUnits &units = second ? down : gated;
            if (second && !(ok = moe_act_ready(s))) break;
            MoeWalk w(units);
            while (w.left > 0 && ok) {
                const uint32_t run = w.run(units);
                const int cols = second ? (s.first[w.expert + 1] - s.first[w.expert] + 15) / 16 * 32 : p.pad;   // of both terms
                const uint32_t idesc = tc_idesc_bf16(128, 16) + (static_cast<uint32_t>((cols - 16) >> 3) << 17);
                const uint32_t d = tmem + buf * kMoeAcc;
                if (!pair_wait(&s.acc_empty[buf], acc_phase, kWaitLimitNs)) {
                    ok = false;
                    break;
                }
                for (uint32_t c = 0; c < run; ++c) {
                    if (!pair_wait(&s.weights_full[st], phase, kWaitLimitNs) || !pair_wait(&s.tokens_full[st], phase, kWaitLimitNs)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint64_t ad = a0 + static_cast<uint32_t>(st) * (stage_bytes >> 4), bd = ad + (kMoeUnit >> 4);
                    if (elect_one()) {
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk) tc_mma_bf16(d, ad + 2 * kk, bd + 2 * kk, idesc, c > 0 || kk > 0);
                        tc_commit(&s.empty[st]);
                        if (c == run - 1) tc_commit(&s.acc_full[buf]);
                    }
                    __syncwarp();
                    if (++st == p.stages) {
                        st = 0;
                        phase ^= 1;
                    }
                }
                w.left -= run;
                w.next_tile(units);
                buf ^= 1;
                if (buf == 0) acc_phase ^= 1;
            }
        }
        // every product issued has ended before the tensor memory is given back
        if (elect_one()) tc_commit(&s.done);
        __syncwarp();
        if (!pair_wait(&s.done, 0, kWaitLimitNs)) ok = false;
    } else if (warp >= kMoeSum) {
        const int sums = kMoeWarps - kMoeSum, me = warp - kMoeSum;
        if (moe_choose_all(p) && me >= 4) {   // read after the barriers below
            moe_weigh(p, s, 0, p.T, me - 4, 4);
            __syncwarp();
            if (blockIdx.x == 0 && p.weights)
                for (int t = me - 4; t < p.T; t += 4)
                    if (lane < p.top_k) p.weights[t * p.top_k + lane] = s.weight[t * p.top_k + lane];
        }
        uint32_t buf = 0, acc_phase = 0;
        for (int second = 0; second < 2 && ok; ++second) {
            const MoeUnits &units = second ? down : gated;
            if (me < 4) {
                const uint32_t lanes = tmem + (static_cast<uint32_t>(me * 32) << 16);
                const int row = me * 32 + lane;
                MoeWalk w(units);
                while (w.left > 0 && ok) {
                    const uint32_t run = w.run(units);
                    const bool whole = w.chunk == 0;   // the tile begins here
                    const int first = s.first[w.expert], count = s.first[w.expert + 1] - first;
                    ok = __all_sync(0xffffffffu, pair_wait(&s.acc_full[buf], acc_phase, 4 * kWaitLimitNs));
                    if (!second && units.whole) {   // the four warps meet below: they go on together, or none does
                        if (!ok) s.tile_failed = 1;   // the block's only tile of this phase
                        bar_sync_named(2, 128);
                        ok = *reinterpret_cast<volatile uint32_t *>(&s.tile_failed) == 0;
                    }
                    if (!ok) break;
                    tc_fence_after();
                    float *carry = p.carry + static_cast<int64_t>(blockIdx.x) * p.pad * 128 + row;
                    if (!second && units.whole) {
                        // g lies in the first two warps, u in the others: exchanged 16 columns at a time
                        const uint64_t mask = s.mask[s.expert[w.expert]];
                        const int n = static_cast<int>(w.tile) * 64 + (row & 63);
                        float *other = reinterpret_cast<float *>(s.sums) + (row & 63);
                        int at = first;
                        for (int c = 0; c < p.pad; c += 16) {
                            const uint32_t m = static_cast<uint32_t>(mask >> c) & 0xffffu;
                            if (m == 0) continue;
                            float v[16];
                            __syncwarp();
                            tmem_ld16(lanes + buf * kMoeAcc + static_cast<uint32_t>(c), v);
                            if (row >= 64) {
#pragma unroll
                                for (int i = 0; i < 16; ++i) other[i * 64] = v[i];
                            }
                            bar_sync_named(2, 128);
                            if (row < 64) {
#pragma unroll
                                for (int i = 0; i < 16; ++i)
                                    if (m >> i & 1u) {
                                        if (n < p.N) {
                                            uint16_t hi, lo;
                                            moe_act(v[i], other[i * 64], hi, lo);
                                            uint16_t *dst = p.act + at * p.act_ld + n;
                                            *dst = hi;
                                            dst[p.act_rows * p.act_ld] = lo;
                                        }
                                        ++at;
                                    }
                            }
                            bar_sync_named(2, 128);
                        }
                    } else if (!second) {
                        const uint64_t mask = s.mask[s.expert[w.expert]];
                        const int n = static_cast<int>(w.tile) * 64 + (row & 63);
                        float *dst = p.gu + first * (2 * static_cast<int64_t>(p.N)) + (row >> 6) * p.N + n;
                        int at = 0;
                        for (int c = 0; c < p.pad; c += 16) {
                            const uint32_t m = static_cast<uint32_t>(mask >> c) & 0xffffu;
                            if (m == 0) continue;
                            float v[16];
                            __syncwarp();
                            tmem_ld16(lanes + buf * kMoeAcc + static_cast<uint32_t>(c), v);
#pragma unroll
                            for (int i = 0; i < 16; ++i) {
                                if (m >> i & 1u) {
                                    if (!whole)
                                        __stcg(carry + at * 128, v[i]);
                                    else if (n < p.N)
                                        __stcg(dst + at * (2 * static_cast<int64_t>(p.N)), v[i]);
                                    ++at;
                                }
                            }
                        }
                    } else {
                        const int k = static_cast<int>(w.tile) * 128 + row;
                        float *dst = p.y + first * static_cast<int64_t>(p.K) + k;
                        for (int c = 0; c < count; c += 16) {
                            float v[16], x[16];
                            __syncwarp();
                            tmem_ld16(lanes + buf * kMoeAcc + static_cast<uint32_t>(c), v);
                            tmem_ld16(lanes + buf * kMoeAcc + static_cast<uint32_t>((count + 15) / 16 * 16 + c), x);
#pragma unroll
                            for (int i = 0; i < 16; ++i) v[i] += x[i];
#pragma unroll
                            for (int i = 0; i < 16; ++i) {
                                if (c + i < count) {
                                    if (!whole)
                                        __stcg(carry + (c + i) * 128, v[i]);
                                    else if (k < p.K)
                                        __stcg(dst + (c + i) * static_cast<int64_t>(p.K), v[i]);
                                }
                            }
                        }
                    }
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&s.acc_empty[buf]);
                    w.left -= run;
                    w.next_tile(units);
                    buf ^= 1;
                    if (buf == 0) acc_phase ^= 1;
                }
            }
            if (!ok) s.failed = 1;
            if (!second && units.whole) fence_proxy_async_all();   // the activation is read by copies
            bar_sync_named(1, sums * 32);
            if (me == 0 && lane == 0) {
                grid_arrive(p.counters + 1 + 2 * second);   // after a failure too: the others need not wait
                if (!grid_wait(p.counters + 1 + 2 * second, 2 * kWaitLimitNs)) s.failed = 1;
                s.phase_failed = *reinterpret_cast<volatile uint32_t *>(&s.failed);
            }
            bar_sync_named(1, sums * 32);
            ok = *reinterpret_cast<volatile uint32_t *>(&s.phase_failed) == 0;
            if (!second && units.whole) {
                if (me == 0 && lane == 0) {
                    fence_proxy_async_all();
                    mbar_arrive(&s.act_ready);
                }
            } else if (!second) {
                // 4: the activation; a warp per slot and tile of 64 columns
                const int slots = s.first[s.active];
                for (uint32_t i = blockIdx.x + gridDim.x * static_cast<uint32_t>(me); ok && i < static_cast<uint32_t>(slots) * units.tiles;
                     i += gridDim.x * static_cast<uint32_t>(sums)) {
                    const uint32_t slot = i / units.tiles, tile = i - slot * units.tiles;
                    const int at = s.of_slot[slot], col = static_cast<int>(slot) - s.first[at];
                    const uint32_t u0 = (static_cast<uint32_t>(at) * units.tiles + tile) * units.chunks;
                    const uint32_t b0 = moe_owner(units, u0), b1 = moe_owner(units, u0 + units.chunks - 1);
                    const int n = static_cast<int>(tile) * 64 + lane * 2;
                    if (n >= p.N) continue;   // N is even: both columns exist, or none
                    const float *src = p.gu + slot * (2 * static_cast<int64_t>(p.N)) + n;
                    float2 g = __ldcg(reinterpret_cast<const float2 *>(src)), u = __ldcg(reinterpret_cast<const float2 *>(src + p.N));
                    const auto part = [&](uint32_t b, int up) {
                        const float *q = p.carry + (static_cast<int64_t>(b) * p.pad + col) * 128 + up * 64 + lane * 2;
                        return b <= b1 ? __ldcg(reinterpret_cast<const float2 *>(q)) : make_float2(0.0f, 0.0f);
                    };
                    for (uint32_t b = b0 + 1; b <= b1; b += 2) {   // two on the way together
                        const float2 x = part(b, 0), z = part(b, 1), x2 = part(b + 1, 0), z2 = part(b + 1, 1);
                        g = make_float2(g.x + x.x + x2.x, g.y + x.y + x2.y);
                        u = make_float2(u.x + z.x + z2.x, u.y + z.y + z2.y);
                    }
                    uint16_t h0, h1, l0, l1;
                    moe_act(g.x, u.x, h0, l0);
                    moe_act(g.y, u.y, h1, l1);
                    uint16_t *dst = p.act + slot * p.act_ld + n;
                    *reinterpret_cast<uint32_t *>(dst) = h0 | static_cast<uint32_t>(h1) << 16;
                    *reinterpret_cast<uint32_t *>(dst + p.act_rows * p.act_ld) = l0 | static_cast<uint32_t>(l1) << 16;
                }
                fence_proxy_async_all();
                bar_sync_named(1, sums * 32);
                if (me == 0 && lane == 0) {
                    grid_arrive(p.counters + 2);
                    if (!grid_wait(p.counters + 2, 2 * kWaitLimitNs)) s.failed = 1;
                    s.phase_failed = *reinterpret_cast<volatile uint32_t *>(&s.failed);
                    fence_proxy_async_all();
                    mbar_arrive(&s.act_ready);
                }
                bar_sync_named(1, sums * 32);
                ok = *reinterpret_cast<volatile uint32_t *>(&s.phase_failed) == 0;
            } else {
                // 6: the weighted sum of a token's 128 columns: a team of warps, each of which takes
                // every team-th expert, four of them at a time
                const uint32_t items = static_cast<uint32_t>(p.T) * units.tiles;
                const uint32_t team = items <= gridDim.x ? 8u : items <= 2 * gridDim.x ? 4u : items <= 4 * gridDim.x ? 2u : 1u;
                const uint32_t mine = static_cast<uint32_t>(me) / team, place = static_cast<uint32_t>(me) % team;
                static_assert(kMoeWarps - kMoeSum == 8, "teams");
                for (uint32_t i = blockIdx.x + gridDim.x * mine; ok && i < items; i += gridDim.x * (8 / team)) {
                    const uint32_t t = i / units.tiles, tile = i - t * units.tiles;
                    const int k = static_cast<int>(tile) * 128 + lane * 4;
                    const bool in = k < p.K;   // K is a multiple of 8
                    float4 sum = make_float4(0, 0, 0, 0);
                    for (uint32_t j0 = place; j0 < static_cast<uint32_t>(p.top_k); j0 += 4 * team) {
                        float4 v[4], x[4];
                        float c[4];
                        uint32_t b0[4], b1[4];
                        int col[4];
#pragma unroll
                        for (int h = 0; h < 4; ++h) {
                            const uint32_t j = j0 + h * team;
                            const bool has = in && j < static_cast<uint32_t>(p.top_k);
                            const int at = static_cast<int>(t) * p.top_k + static_cast<int>(has ? j : place);
                            const int e = s.id[at], w = s.where[e];
                            col[h] = __popcll(s.mask[e] & ((1ull << t) - 1));
                            c[h] = has ? s.weight[at] : 0.0f;
                            const uint32_t u0 = (static_cast<uint32_t>(w) * units.tiles + tile) * units.chunks;
                            b0[h] = moe_owner(units, u0);
                            b1[h] = moe_owner(units, u0 + units.chunks - 1);
                            const float4 none = make_float4(0, 0, 0, 0);
                            v[h] = has ? __ldcg(reinterpret_cast<const float4 *>(p.y + (s.first[w] + col[h]) * static_cast<int64_t>(p.K) + k)) : none;
                            x[h] = has && b1[h] > b0[h]
                                       ? __ldcg(reinterpret_cast<const float4 *>(p.carry + (static_cast<int64_t>(b0[h] + 1) * p.pad + col[h]) * 128 + lane * 4))
                                       : none;
                            if (!has) b1[h] = b0[h];
                        }
#pragma unroll
                        for (int h = 0; h < 4; ++h) {
                            v[h] = make_float4(v[h].x + x[h].x, v[h].y + x[h].y, v[h].z + x[h].z, v[h].w + x[h].w);
                            for (uint32_t b = b0[h] + 2; b <= b1[h]; ++b) {
                                const float4 z = __ldcg(reinterpret_cast<const float4 *>(p.carry + (static_cast<int64_t>(b) * p.pad + col[h]) * 128 + lane * 4));
                                v[h] = make_float4(v[h].x + z.x, v[h].y + z.y, v[h].z + z.z, v[h].w + z.w);
                            }
                            sum.x = fmaf(c[h], v[h].x, sum.x);
                            sum.y = fmaf(c[h], v[h].y, sum.y);
                            sum.z = fmaf(c[h], v[h].z, sum.z);
                            sum.w = fmaf(c[h], v[h].w, sum.w);
                        }
                    }
                    if (team > 1) {   // one item per team and phase: no sum is written twice
                        s.sums[me][lane] = sum;
                        bar_sync_named(2 + static_cast<int>(mine), static_cast<int>(team) * 32);
                        if (place != 0) break;
                        for (uint32_t h = 1; h < team; ++h) {
                            const float4 z = s.sums[me + h][lane];
                            sum = make_float4(sum.x + z.x, sum.y + z.y, sum.z + z.z, sum.w + z.w);
                        }
                    }
                    if (in) *reinterpret_cast<uint2 *>(p.out + t * p.ldo + k) = make_uint2(pack_bf16x2(sum.x, sum.y), pack_bf16x2(sum.z, sum.w));
                }
            }
        }
    }
    if (!ok) {
        s.failed = 1;
        atomicExch(&g_dense_error, kErrTimeout);
    }
    tc_fence_before();
    __syncthreads();
    __syncwarp();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, kMoeCols);
    }
    if (threadIdx.x == 0) {
        if (s.failed != 0) {
            grid_fail(p.counters);
        } else {
            // the last block to leave: everyone has passed every barrier
            const uint32_t left = add_acq_rel_gpu(p.counters + 4, 1u);
            if (left == gridDim.x - 1) {
                for (int i = 0; i < kMoeCounters; ++i) p.counters[i] = 0;
            } else if (left >= gridDim.x) {
                atomicExch(&g_dense_error, kErrTimeout);
                grid_fail(p.counters);
            }
        }
    }
}

}  // namespace mbglu
