// pair_gemm.cuh -- the pipeline of the tensor-core products on CTA pairs, and
// the bf16 kernel on it: both projections of the gated block with their
// epilogues, and the three gradient products.
//
// A cluster of two CTAs (an SM pair) owns a tile of 256 rows x 256 accumulator
// columns; tcgen05.mma of cta_group::2 reads 128 rows of A and 128 of B from
// each SM's shared memory, so an operand byte is brought in once per pair and
// each SM's shared memory feeds twice the arithmetic that it would alone.  One
// persistent cluster per SM pair walks the tiles; roles per CTA (384 threads):
//   warp 0      tensor copies: per stage 16 KB of A and 16 KB of B
//               (64 bf16 or 128 e4m3 of the inner dimension), 6 stages;
//               both CTAs' copies count on the even CTA's barrier
//   warp 1      owns the tensor memory -- two buffers of 256 columns, so that a
//               tile's epilogue runs under the next tile's products -- and, in
//               the even CTA, issues the MMAs
//   warps 4-11  epilogue: warp w reads lanes 32 (w % 4).., the first or second
//               half of the columns
// A gated tile holds 128 gate and 128 up columns of the same outputs: the even
// CTA brings the gate rows, the odd one the up rows, and g and u of one output
// meet in one thread.
//
// Tiles run along rows first within groups of `group` row tiles, so the tiles
// in flight share operands in L2.  Every wait is bounded; after one gives up
// each role runs its loops to the end without touching memory.
#pragma once

#include "dense_common.cuh"
#include "tc_pair.cuh"

namespace mbglu {

constexpr int kPairThreads = 384;
constexpr int kPairEpilogue = 4;                            // the first of the eight epilogue warps
constexpr int kPairStages = 6;
constexpr int kPairTile = 256;
constexpr uint32_t kPairOperand = 16384;                   // one operand's bytes per stage and CTA
constexpr uint32_t kPairStage = 2 * kPairOperand;
constexpr uint32_t kPairHeader = 4096;                     // barriers, tensor-memory address, the epilogue's exchange
constexpr uint32_t kPairExchange = 1024;                   // offset of the exchange within the header
constexpr uint32_t kPairRowBufs = 8 * kRowBuf * 4;         // the epilogue warps' buffers for unaligned rows
constexpr uint32_t kPairSmem = kPairHeader + kPairStages * kPairStage + kPairRowBufs + 1024;   // + alignment
constexpr uint32_t kPairCols = 512;

// How a tile's operands are chosen.
enum PairMode {
    kPairDual = 0,    // b[0] rows (even CTA) and b[1] rows (odd CTA) of the same 128 outputs
    kPairSum = 1,     // a[0] b[0] + a[1] b[1] (a[1], b[1] after nchunk0 chunks)
    kPairStack = 2    // nout products a[o] b[0]
};

struct PairMaps {
    TensorMap a[2], b[2];
};

struct PairPlan {
    int rows, cols;          // of one output
    int mt, nt, nout;        // row tiles, column tiles, outputs
    int whole;               // tiles done whole: full rounds over the SM pairs
    int rest, splits;        // the others, each in `splits` ranges of the inner dimension
    int ntiles;              // whole + rest splits: work items
    int group;
    int nchunk0, nchunk;     // chunks of the first product, of all
};

struct PairTileAt {
    int o, mi, ni, c0, c1;
    int slot;   // where a range's partial sums go, or -1
};

// Tile `t` of the outputs: rows first within groups of row tiles.
__host__ __device__ inline void pair_place(const PairPlan &p, int t, PairTileAt &x)
{
    const int per = p.mt * p.nt;
    x.o = t / per;
    t -= x.o * per;
    const int g = t / (p.group * p.nt), first = g * p.group;
    const int gm = p.mt - first < p.group ? p.mt - first : p.group;
    t -= first * p.nt;
    x.mi = first + t % gm;
    x.ni = t / gm;
}

__host__ __device__ inline PairTileAt pair_tile(const PairPlan &p, int t)
{
    PairTileAt x;
    x.slot = t < p.whole ? -1 : t - p.whole;
    x.c0 = 0;
    x.c1 = p.nchunk;
    if (x.slot >= 0) {
        const int split = x.slot / p.rest;
        t = p.whole + x.slot % p.rest;
        x.c0 = static_cast<int>(static_cast<int64_t>(p.nchunk) * split / p.splits);
        x.c1 = static_cast<int>(static_cast<int64_t>(p.nchunk) * (split + 1) / p.splits);
        if (p.splits == 1) x.slot = -1;
    }
    pair_place(p, t, x);
    return x;
}

// fp32 values of one slot: a tile, row by row
constexpr int64_t kPairSlot = static_cast<int64_t>(kPairTile) * kPairTile;

struct PairShared {
    uint64_t *full, *empty, *acc_full, *acc_empty;
    uint32_t *slot;
    unsigned char *stages;
    uint32_t *row_bufs;
    float *exchange;
};

__device__ __forceinline__ PairShared pair_shared(unsigned char *raw)
{
    unsigned char *base = raw + ((1024u - (smem_addr(raw) & 1023u)) & 1023u);
    PairShared s;
    s.full = reinterpret_cast<uint64_t *>(base);
    s.empty = s.full + kPairStages;
    s.acc_full = s.empty + kPairStages;
    s.acc_empty = s.acc_full + 2;
    s.slot = reinterpret_cast<uint32_t *>(s.acc_empty + 2);
    s.exchange = reinterpret_cast<float *>(base + kPairExchange);
    s.stages = base + kPairHeader;
    s.row_bufs = reinterpret_cast<uint32_t *>(s.stages + kPairStages * kPairStage);
    return s;
}

// Barriers and tensor memory; returns the tensor-memory address.
__device__ __forceinline__ uint32_t pair_setup(const PairShared &s, int warp)
{
    if (threadIdx.x == 0) {
        for (int i = 0; i < kPairStages; ++i) {
            mbar_init(&s.full[i], 1);
            mbar_init(&s.empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s.acc_full[i], 1);
            mbar_init(&s.acc_empty[i], 16);   // the epilogue warps of both CTAs
        }
        fence_mbar_init();
    }
    if (warp == 1) {
        pair_tmem_alloc(s.slot, kPairCols);
        pair_tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    __syncwarp();
    cluster_sync();   // the other CTA's barriers and tensor memory exist
    tc_fence_after();
    return __shfl_sync(0xffffffffu, *s.slot, 0);
}

__device__ __forceinline__ void pair_teardown(int warp, uint32_t tmem)
{
    tc_fence_before();
    __syncthreads();
    __syncwarp();
    cluster_sync();   // both CTAs have read their accumulators and sent their arrivals
    if (warp == 1) {
        tc_fence_after();
        pair_tmem_dealloc(tmem, kPairCols);
    }
}

// Warp 0.  CK: elements of the inner dimension per chunk.
template <int MODE, bool A_MN, bool B_MN, int CK>
__device__ __forceinline__ bool pair_produce(const PairPlan &p, const PairMaps &maps, const PairShared &s, uint32_t rank)
{
    // this warp's instructions stand between a freed stage and its next copies,
    // so the ring is walked by a stage number and a phase bit, without divisions
    int st = 0;
    uint32_t phase = 1;   // of empty[]: the first round's stages are free
    bool ok = true;
    uint32_t filled = 0;  // up to kPairStages
    const uint32_t full0 = map_to_rank(s.full, 0);
    for (int t = static_cast<int>(blockIdx.x >> 1); t < p.ntiles && ok; t += static_cast<int>(gridDim.x >> 1)) {
        const PairTileAt x = pair_tile(p, t);
        const int arow = x.mi * kPairTile + static_cast<int>(rank) * 128;
        const int brow = MODE == kPairDual ? x.ni * 128 : x.ni * kPairTile + static_cast<int>(rank) * 128;
        for (int c = x.c0; c < x.c1; ++c) {
            if (!pair_wait(&s.empty[st], phase, kWaitLimitNs)) {
                ok = false;
                break;
            }
            const bool second = MODE == kPairSum && c >= p.nchunk0;
            const int k = (second ? c - p.nchunk0 : c) * CK;
            const TensorMap *ma = &maps.a[MODE == kPairSum ? second : MODE == kPairStack ? x.o : 0];
            const TensorMap *mb = &maps.b[MODE == kPairSum ? second : MODE == kPairDual ? static_cast<int>(rank) : 0];
            unsigned char *da = s.stages + st * kPairStage, *db = da + kPairOperand;
            const uint32_t bar = full0 + static_cast<uint32_t>(st) * 8u;
            if (elect_one()) {
                if (rank == 0) mbar_arrive_expect_tx(&s.full[st], 2 * kPairStage);
                if (A_MN) {
                    pair_load_2d(da, ma, arow, k, bar);
                    pair_load_2d(da + kPairBoxBytes, ma, arow + 64, k, bar);
                } else {
                    pair_load_2d(da, ma, k, arow, bar);
                }
                if (B_MN) {
                    pair_load_2d(db, mb, brow, k, bar);
                    pair_load_2d(db + kPairBoxBytes, mb, brow + 64, k, bar);
                } else {
                    pair_load_2d(db, mb, k, brow, bar);
                }
            }
            __syncwarp();
            filled += filled < kPairStages;
            if (++st == kPairStages) {
                st = 0;
                phase ^= 1;
            }
        }
    }
    // every copy of this CTA has landed and been read, and every arrival on
    // this CTA's barriers has come, before it may leave: the last round's
    // stages, oldest first
    for (uint32_t i = 0; i < filled; ++i) {
        int at = st - static_cast<int>(filled - i);
        const uint32_t ph = at < 0 ? phase : phase ^ 1;   // filled in the round before this one, or in this
        if (at < 0) at += kPairStages;
        if (!pair_wait(&s.empty[at], ph, kWaitLimitNs)) ok = false;
    }
    return ok;
}

// Warp 1 of the even CTA.  PER_CHUNK: each chunk is a sum of its
// own in the next buffer (block-scaled operands), else a tile is.
template <bool A_MN, bool B_MN, bool E4M3, bool PER_CHUNK>
__device__ __forceinline__ bool pair_multiply(const PairPlan &p, const PairShared &s, uint32_t tmem)
{
    constexpr uint32_t idesc = E4M3 ? pair_idesc_e4m3() : pair_idesc_bf16(A_MN, B_MN);
    const uint64_t a0 = A_MN ? smem_desc_mn_sw128(s.stages) : smem_desc_sw128(s.stages);
    const uint64_t b0 = B_MN ? smem_desc_mn_sw128(s.stages + kPairOperand) : smem_desc_sw128(s.stages + kPairOperand);
    int st = 0;
    uint32_t phase = 0, buf = 0, acc_phase = 1;   // of full[], of acc_empty[] (both buffers start free)
    for (int t = static_cast<int>(blockIdx.x >> 1); t < p.ntiles; t += static_cast<int>(gridDim.x >> 1)) {
        const PairTileAt x = pair_tile(p, t);
        for (int c = x.c0; c < x.c1; ++c) {
            if ((PER_CHUNK || c == x.c0) && !pair_wait(&s.acc_empty[buf], acc_phase, kWaitLimitNs)) return false;
            if (!pair_wait(&s.full[st], phase, kWaitLimitNs)) return false;
            tc_fence_after();
            const uint64_t ad = a0 + static_cast<uint32_t>(st) * (kPairStage >> 4);
            const uint64_t bd = b0 + static_cast<uint32_t>(st) * (kPairStage >> 4);
            const uint32_t d = tmem + buf * kPairTile;
            if (elect_one()) {
#pragma unroll
                for (int kk = 0; kk < 4; ++kk) {   // 16 bf16 or 32 e4m3 each
                    const bool acc = kk > 0 || (!PER_CHUNK && c > x.c0);
                    const uint64_t a = ad + (A_MN ? 128 : 2) * kk, b = bd + (B_MN ? 128 : 2) * kk;
                    if (E4M3)
                        pair_mma_e4m3(d, a, b, idesc, acc);
                    else
                        pair_mma_bf16(d, a, b, idesc, acc);
                }
                pair_commit(&s.empty[st]);
                if (PER_CHUNK || c == x.c1 - 1) pair_commit(&s.acc_full[buf]);
            }
            __syncwarp();
            if (++st == kPairStages) {
                st = 0;
                phase ^= 1;
            }
            if (PER_CHUNK || c == x.c1 - 1) {
                buf ^= 1;
                if (buf == 0) acc_phase ^= 1;
            }
        }
    }
    return true;
}

enum PairKind { kPairGlu = 0, kPairGrad = 1, kPairPlain = 2 };

struct PairParams {
    PairPlan plan;
    int mode;
    uint16_t *out[2];
    int64_t ldo[2];
    int out_align[2];
    float *gu;               // g and u, [rows][2 cols], or null
    int64_t ldgu;
    int gu_align, gu_align_u;
    const uint16_t *dout;
    int64_t ldd;
    int dout_align;
    float *part;             // ranges' partial sums, kPairSlot each
};

template <int EPI, int MODE, bool A_MN, bool B_MN>
__global__ void __launch_bounds__(kPairThreads, 1) pair_gemm_kernel(const PairParams p, const __grid_constant__ PairMaps maps)
{
    extern __shared__ unsigned char pair_raw[];
    const PairShared s = pair_shared(pair_raw);
    const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();
    const uint32_t tmem = pair_setup(s, warp);
    grid_dependency_wait();
    grid_launch_dependents();
    bool ok = true;

    if (warp == 0) {
        ok = pair_produce<MODE, A_MN, B_MN, 64>(p.plan, maps, s, rank);
    } else if (warp == 1) {
        if (rank == 0) ok = pair_multiply<A_MN, B_MN, false, false>(p.plan, s, tmem);
    } else if (warp >= kPairEpilogue) {
        const int q = warp & 3, half = (warp - kPairEpilogue) >> 2;
        const uint32_t lanes = tmem + (static_cast<uint32_t>(q * 32) << 16);
        uint32_t v = 0;
        for (int t = static_cast<int>(blockIdx.x >> 1); t < p.plan.ntiles; t += static_cast<int>(gridDim.x >> 1), ++v) {
            const PairTileAt x = pair_tile(p.plan, t);
            const int buf = static_cast<int>(v & 1);
            const int64_t m = static_cast<int64_t>(x.mi) * kPairTile + rank * 128 + q * 32;   // the warp's first row
            const int rows = static_cast<int>(min(static_cast<int64_t>(32), p.plan.rows - m));
            uint32_t *buf32 = s.row_bufs + (warp - kPairEpilogue) * kRowBuf;
            if (ok) ok = __all_sync(0xffffffffu, pair_wait(&s.acc_full[buf], (v >> 1) & 1, kWaitLimitNs));
            tc_fence_after();
            const uint32_t acc = lanes + static_cast<uint32_t>(buf) * kPairTile;
            if constexpr (MODE == kPairDual) {
#pragma unroll 1
                for (int j = 0; j < 2; ++j) {
                    const int c = half * 64 + j * 32;
                    const int n = x.ni * 128 + c, valid = p.plan.cols - n;
                    uint32_t g[32], u[32];
                    tmem_ld32(acc + static_cast<uint32_t>(c), g);
                    tmem_ld32(acc + 128u + static_cast<uint32_t>(c), u);
                    float d[32];
                    if (EPI == kPairGrad && rows > 0 && valid > 0) warp_load_bf16(buf32, p.dout + m * p.ldd + n, p.ldd, d, rows, valid, p.dout_align);
                    tmem_wait_ld(g, u);
                    if (j == 1) {   // the buffer is read
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) pair_arrive(map_to_rank(&s.acc_empty[buf], 0));
                    }
                    if (!ok || rows <= 0 || valid <= 0) continue;   // the whole warp
                    uint32_t w[16], w2[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const float g0 = __uint_as_float(g[2 * i]), g1 = __uint_as_float(g[2 * i + 1]);
                        const float u0 = __uint_as_float(u[2 * i]), u1 = __uint_as_float(u[2 * i + 1]);
                        if (EPI == kPairGrad) {
                            float dg0, du0, dg1, du1;
                            glu_gradients(g0, u0, d[2 * i], dg0, du0);
                            glu_gradients(g1, u1, d[2 * i + 1], dg1, du1);
                            w[i] = pack_bf16x2(dg0, dg1);
                            w2[i] = pack_bf16x2(du0, du1);
                        } else if (p.mode == 0) {
                            w[i] = pack_bf16x2(silu_short(g0) * u0, silu_short(g1) * u1);
                        } else {
                            w[i] = glu_hf_short(g0, u0) | (glu_hf_short(g1, u1) << 16);
                        }
                    }
                    warp_store_bf16(buf32, p.out[0] + m * p.ldo[0] + n, p.ldo[0], w, rows, valid, p.out_align[0]);
                    if (EPI == kPairGrad) warp_store_bf16(buf32, p.out[1] + m * p.ldo[1] + n, p.ldo[1], w2, rows, valid, p.out_align[1]);
                    if (EPI == kPairGlu && p.gu) {
                        warp_store_f32(buf32, p.gu + m * p.ldgu + n, p.ldgu, g, rows, valid, p.gu_align);
                        warp_store_f32(buf32, p.gu + m * p.ldgu + p.plan.cols + n, p.ldgu, u, rows, valid, p.gu_align_u);
                    }
                }
            } else {
#pragma unroll 1
                for (int j = 0; j < 4; ++j) {
                    const int c = half * 128 + j * 32;
                    const int n = x.ni * kPairTile + c, valid = p.plan.cols - n;
                    uint32_t r[32];
                    tmem_ld32(acc + static_cast<uint32_t>(c), r);
                    tmem_wait_ld(r);
                    if (j == 3) {
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) pair_arrive(map_to_rank(&s.acc_empty[buf], 0));
                    }
                    if (!ok || rows <= 0 || valid <= 0) continue;   // the whole warp
                    if (x.slot >= 0) {
                        warp_store_f32(buf32, p.part + x.slot * kPairSlot + (rank * 128 + q * 32) * kPairTile + c, kPairTile, r, rows, 32, 2);
                    } else {
                        uint32_t w[16];
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            w[i] = pack_bf16x2(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1]));
                        const int o = MODE == kPairStack ? x.o : 0;
                        warp_store_bf16(buf32, p.out[o] + m * p.ldo[o] + n, p.ldo[o], w, rows, valid, p.out_align[o]);
                    }
                }
            }
        }
    }
    if (!ok) atomicExch(&g_dense_error, kErrTimeout);
    pair_teardown(warp, tmem);
}

struct PairJoin {
    PairPlan plan;
    const float *part;
    uint16_t *out[2];
    int64_t ldo[2];
    int vec[2];              // rows of the output lie on 8 bytes
};

// The split tiles: out = bf16(sum of their ranges' partial sums, in order).  A
// block of 256 threads takes 4 rows of a tile, 4 columns per thread.
static __global__ void __launch_bounds__(256) pair_join_kernel(const PairJoin p)
{
    grid_dependency_wait();
    grid_launch_dependents();
    const int tile = blockIdx.x >> 6, r = (blockIdx.x & 63) * 4 + (threadIdx.x >> 6), c = (threadIdx.x & 63) * 4;
    PairTileAt x;
    pair_place(p.plan, p.plan.whole + tile, x);
    const int64_t m = static_cast<int64_t>(x.mi) * kPairTile + r;
    const int n = x.ni * kPairTile + c, valid = p.plan.cols - n;
    if (m >= p.plan.rows || valid <= 0) return;
    const float *q = p.part + tile * kPairSlot + r * kPairTile + c;
    float4 a = make_float4(0, 0, 0, 0);
#pragma unroll 4
    for (int s = 0; s < p.plan.splits; ++s) {
        const float4 b = __ldcs(reinterpret_cast<const float4 *>(q + static_cast<int64_t>(s) * p.plan.rest * kPairSlot));
        a.x += b.x;
        a.y += b.y;
        a.z += b.z;
        a.w += b.w;
    }
    uint16_t *o = p.out[x.o] + m * p.ldo[x.o] + n;
    const uint2 w = make_uint2(pack_bf16x2(a.x, a.y), pack_bf16x2(a.z, a.w));
    if (p.vec[x.o] && valid >= 4) {
        *reinterpret_cast<uint2 *>(o) = w;
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (i < valid) o[i] = static_cast<uint16_t>((i < 2 ? w.x : w.y) >> ((i & 1) * 16));
    }
}

}  // namespace mbglu
