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

// Ranges of the inner dimension (of `chunks` stages): where 256 x 256 tiles
// leave most SM pairs idle, as many as fill them, each of at least 8 stages.
// From the sizes alone, so that the sum's order does not depend on the device.
inline int pair_splits(int rows, int cols, int64_t chunks)
{
    const int64_t tiles = static_cast<int64_t>(ceil_div(rows, mbglu::kPairTile)) * ceil_div(cols, mbglu::kPairTile);
    return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>({kPairs / tiles, chunks / 8, 16})));
}

// Row stride of the partial sums, fp32: rows start on 32 bytes.
inline int64_t part_width(int cols) { return (static_cast<int64_t>(cols) + 7) / 8 * 8; }

inline mbglu::PairPlan pair_plan(int rows, int cols, int tile_cols, int nout, int nchunk0, int nchunk, int splits)
{
    mbglu::PairPlan p = {};
    p.rows = rows;
    p.cols = cols;
    p.mt = ceil_div(rows, mbglu::kPairTile);
    p.nt = ceil_div(cols, tile_cols);
    p.nout = nout;
    p.splits = splits;
    p.ntiles = p.mt * p.nt * nout * splits;
    p.group = 8;
    p.nchunk0 = nchunk0;
    p.nchunk = nchunk;
    return p;
}

inline mbglu_status launch_join(const float *part, int splits, int rows, int cols, uint16_t *out, int64_t ldo,
                                cudaStream_t stream)
{
    const int vec = cols % 4 == 0 && aligned(out, 8) && ldo % 4 == 0;
    const int64_t work = static_cast<int64_t>(rows) * (vec ? cols / 4 : cols);
    Launch l(dim3(static_cast<unsigned>(std::min<int64_t>((work + 255) / 256, 1 << 20))), 256, 0, stream);
    return launched(cudaLaunchKernelEx(&l.cfg, mbglu::pair_join_kernel, part, splits, rows, cols, part_width(cols), out, ldo, vec));
}

}  // namespace mbglu_host
