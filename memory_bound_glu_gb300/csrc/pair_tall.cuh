// pair_tall.cuh -- glu_gemm's forward on CTA pairs with the weights on the MMA's
// 256-row side and the tokens on the other: for batches that fill 256-row tiles
// badly (a chunk of some hundred tokens), and products of few tiles.
//
// A tile is wt outputs x tn tokens, wt a multiple of 16 up to 128, tn of 32 up to
// 256.  The even CTA's rows are the gate and up rows of the first wt / 2 outputs, the
// odd one's those of the others: g lies from lane 0 of a CTA's tensor memory on, u
// from lane 64.  Below 128 outputs the lanes between hold products of whatever the
// stage holds there, and nobody reads them; such tiles are for even rounds (N = 11008
// is 86 tiles of 128, a second round for ten pairs of 76, or 138 of 80).
// A warp of g and the warp that has u of the same outputs swap halves: of 16
// tokens the first works on 8, the second on the others.  Pipeline and roles as
// pair_gemm.cuh.
//
// What bounds it: the weights' bytes up to about 128 tokens (K = 2560, N = 9728 at M =
// 96: 20.8 us, 14.7 of them the bytes at the copy rate), the MMAs beyond (333: 27.9 us,
// the tensor pipe active for 54%), and a call's start and end (4 us) where there are
// few tiles.  The last tile's epilogue is part of that end and bound by its
// instructions: one pointer stepped by a row, and SiLUs apart from the stores, took
// 29.0 to 27.9 us.  Loading the next 16 columns ahead brought nothing.  With g and u
// written as well: 32.1 us at M = 333, in 256-row tiles 36.1.
#pragma once

#include "pair_gemm.cuh"

namespace mbglu {

struct PairTallParams {
    int M, N, nchunk;
    int wt, tn;               // outputs and tokens per tile
    int ttiles, ntiles;       // tiles along the tokens, in all
    int mode;
    uint16_t *out;
    int64_t ldo;
    float *gu;                // g and u, [M][2 N], or null
    int64_t ldgu;
};

// The exchange between two warps: 2 sets x (8 tokens of g, 8 of u) x 32 lanes.
constexpr int kPairSwap = 2 * 16 * 32;
static_assert(4 * kPairSwap * 4 <= kPairRowBufs, "the exchange takes the place of the row buffers");

static __global__ void __launch_bounds__(kPairThreads, 1) pair_tall_kernel(const PairTallParams p, const __grid_constant__ PairMaps maps)
{
    extern __shared__ unsigned char pair_raw[];
    const PairShared s = pair_shared(pair_raw);
    const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
    const int rank = static_cast<int>(cluster_ctarank());
    const uint32_t tmem = pair_setup(s, warp);
    grid_dependency_wait();
    grid_launch_dependents();
    bool ok = true;
    const int first = static_cast<int>(blockIdx.x >> 1), step = static_cast<int>(gridDim.x >> 1);

    if (warp == 0) {
        const uint32_t full0 = map_to_rank(s.full, 0);
        const uint32_t bytes = 2 * (static_cast<uint32_t>(p.wt) * 128u + static_cast<uint32_t>(p.tn) * 64u);   // both CTAs'
        int st = 0, filled = 0;
        uint32_t phase = 1;
        for (int t = first; t < p.ntiles && ok; t += step) {
            const int n0 = t / p.ttiles * p.wt + rank * (p.wt / 2), m0 = t % p.ttiles * p.tn + rank * (p.tn / 2);
            for (int c = 0; c < p.nchunk; ++c) {
                if (!pair_wait(&s.empty[st], phase, kWaitLimitNs)) {
                    ok = false;
                    break;
                }
                unsigned char *d = s.stages + st * kPairStage;
                const uint32_t bar = full0 + static_cast<uint32_t>(st) * 8u;
                if (elect_one()) {
                    if (rank == 0) mbar_arrive_expect_tx(&s.full[st], bytes);
                    pair_load_2d(d, &maps.a[0], c * 64, n0, bar);
                    pair_load_2d(d + kPairOperand / 2, &maps.a[1], c * 64, n0, bar);
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
        // as pair_produce: the last round's stages, oldest first
        for (int i = 0; i < filled; ++i) {
            int at = st - (filled - i);
            const uint32_t ph = at < 0 ? phase : phase ^ 1;
            if (at < 0) at += kPairStages;
            if (!pair_wait(&s.empty[at], ph, kWaitLimitNs)) ok = false;
        }
    } else if (warp == 1) {
        if (rank == 0) {
            const uint32_t idesc = tc_idesc_bf16(256, 256) - (static_cast<uint32_t>((256 - p.tn) >> 3) << 17);
            const uint64_t a0 = smem_desc_sw128(s.stages), b0 = smem_desc_sw128(s.stages + kPairOperand);
            int st = 0;
            uint32_t phase = 0, buf = 0, acc_phase = 1;
            for (int t = first; t < p.ntiles && ok; t += step) {
                for (int c = 0; c < p.nchunk; ++c) {
                    if ((c == 0 && !pair_wait(&s.acc_empty[buf], acc_phase, kWaitLimitNs)) || !pair_wait(&s.full[st], phase, kWaitLimitNs)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint64_t a = a0 + static_cast<uint32_t>(st) * (kPairStage >> 4), b = b0 + static_cast<uint32_t>(st) * (kPairStage >> 4);
                    if (elect_one()) {
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk) pair_mma_bf16(tmem + buf * kPairTile, a + 2 * kk, b + 2 * kk, idesc, kk > 0 || c > 0);
                        pair_commit(&s.empty[st]);
                        if (c == p.nchunk - 1) pair_commit(&s.acc_full[buf]);
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
        const int q = warp & 3, half = (warp - kPairEpilogue) >> 2, side = q >> 1;   // side: 0 has g, 1 has u
        const uint32_t lanes = tmem + (static_cast<uint32_t>(q * 32) << 16) + static_cast<uint32_t>(half * (p.tn / 2));
        const int pairing = half * 2 + (q & 1);
        float *swap = reinterpret_cast<float *>(s.row_bufs) + pairing * kPairSwap + lane;
        uint32_t v = 0, sets = 0;
        for (int t = first; t < p.ntiles; t += step, ++v) {
            const uint32_t buf = v & 1;
            const int row = (q & 1) * 32 + lane;
            const int n = row < p.wt / 2 ? t / p.ttiles * p.wt + rank * (p.wt / 2) + row : p.N;   // p.N: none
            const int m0 = t % p.ttiles * p.tn + half * (p.tn / 2);
            if (ok) ok = __all_sync(0xffffffffu, pair_wait(&s.acc_full[buf], (v >> 1) & 1, kWaitLimitNs));
            tc_fence_after();
            for (int j = 0; j < p.tn / 2; j += 16, ++sets) {
                uint32_t r[16];
                tmem_load(lanes + buf * kPairTile + static_cast<uint32_t>(j), r);
                tmem_wait_ld(r);
                if (j + 16 == p.tn / 2) {   // the buffer is read
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) pair_arrive(map_to_rank(&s.acc_empty[buf], 0));
                }
                if (p.gu) {
                    const int left = n < p.N && ok ? p.M - m0 - j : 0;
                    float *o = p.gu + static_cast<int64_t>(m0 + j) * p.ldgu + (side ? p.N : 0) + n;
#pragma unroll
                    for (int i = 0; i < 16; ++i, o += p.ldgu)
                        if (i < left) *o = __uint_as_float(r[i]);
                }
                // two sets in turn: one is written again only after the barrier that
                // the other warp reaches when it has read it
                float *mine = swap + (sets & 1) * 512 + side * 256, *theirs = swap + (sets & 1) * 512 + (side ^ 1) * 256;
#pragma unroll
                for (int i = 0; i < 8; ++i) mine[i * 32] = __uint_as_float(side ? r[i] : r[8 + i]);
                bar_sync_named(1 + pairing, 64);
                const int m = m0 + j + side * 8, left = n < p.N && ok ? p.M - m : 0;
                uint16_t *o = p.out + static_cast<int64_t>(m) * p.ldo + n;
                float g[8], u[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float x = theirs[i * 32], own = __uint_as_float(side ? r[8 + i] : r[i]);
                    g[i] = side ? x : own;
                    u[i] = side ? own : x;
                }
                uint16_t y[8];
                if (p.mode == 0) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) y[i] = f32_to_bf16(silu_short(g[i]) * u[i]);
                } else {
#pragma unroll
                    for (int i = 0; i < 8; ++i) y[i] = static_cast<uint16_t>(glu_hf_short(g[i], u[i]));
                }
#pragma unroll
                for (int i = 0; i < 8; ++i, o += p.ldo)
                    if (i < left) *o = y[i];
            }
        }
    }
    if (!ok) atomicExch(&g_dense_error, kErrTimeout);
    pair_teardown(warp, tmem);
}

}  // namespace mbglu
