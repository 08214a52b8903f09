// pair_plan.h -- host-side planning of the CTA-pair products: tiles, ranges of
// the inner dimension, operands' alignment, and the join of partial sums.
#pragma once
#include <algorithm>

#include "dense_launch.h"
#include "pair_gemm.cuh"

namespace mbglu_host {

constexpr int kPairs = 76;   // SM pairs of the part: what a split of the inner dimension is planned for

// An operand that tensor copies take: 16-byte aligned rows.
inline bool copyable(const void *p, int64_t ld, int elem) { return aligned(p, 16) && ld * elem % 16 == 0; }

// 2 when every row of elem-byte elements starts on 32 bytes, 1 on 16, else 0
inline int row_align(const void *p, int64_t ld, int elem)
{
    return aligned(p, 32) && ld * elem % 32 == 0 ? 2 : aligned(p, 16) && ld * elem % 16 == 0 ? 1 : 0;
}

// A product's tiles over the SM pairs: full rounds whole; what is left over,
// where it fills at most half of the pairs, in as many ranges of the inner
// dimension as fill them (each of at least 8 stages), if that shortens the
// product by more than the join of the partial sums costs (about 24 stages'
// time, 6 us).  From the sizes alone, so that the order of a sum does not depend
// on the device.  M = 4096, K = 2560, 2 N = 19456: grad_h's 160 tiles and
// their join take 218 us against 277 us in three rounds.
inline mbglu::PairPlan pair_plan(int rows, int cols, int tile_cols, int nout, int nchunk0, int nchunk, bool may_split)
{
    mbglu::PairPlan p = {};
    p.rows = rows;
    p.cols = cols;
    p.mt = ceil_div(rows, mbglu::kPairTile);
    p.nt = ceil_div(cols, tile_cols);
    p.nout = nout;
    p.group = 8;
    p.nchunk0 = nchunk0;
    p.nchunk = nchunk;
    const int tiles = p.mt * p.nt * nout;
    p.whole = tiles;
    p.rest = 0;
    p.splits = 1;
    const int left = tiles % kPairs;
    if (may_split && left > 0) {
        const int s = std::min({kPairs / left, nchunk / 8, 16});
        if (s > 1 && nchunk - nchunk / s >= 24) {
            p.whole = tiles - left;
            p.rest = left;
            p.splits = s;
        }
    }
    p.ntiles = p.whole + p.rest * p.splits;
    return p;
}

// Bytes of the partial sums.
inline int64_t part_bytes(const mbglu::PairPlan &p) { return static_cast<int64_t>(p.rest) * p.splits * mbglu::kPairSlot * 4; }

inline mbglu_status launch_join(const mbglu::PairPlan &plan, const float *part, uint16_t *const out[2], const int64_t ldo[2],
                                cudaStream_t stream)
{
    if (plan.rest == 0) return MBGLU_OK;
    mbglu::PairJoin p = {};
    p.plan = plan;
    p.part = part;
    for (int o = 0; o < plan.nout; ++o) {
        p.out[o] = out[o];
        p.ldo[o] = ldo[o];
        p.vec[o] = aligned(out[o], 8) && ldo[o] % 4 == 0;
    }
    Launch l(dim3(static_cast<unsigned>(plan.rest) * 64), 256, 0, stream);
    return launched(cudaLaunchKernelEx(&l.cfg, mbglu::pair_join_kernel, p));
}

}  // namespace mbglu_host
