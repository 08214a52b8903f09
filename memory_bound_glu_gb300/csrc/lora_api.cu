// lora_api.cu -- products with low-rank adapters of many requests beside the shared
// weights (glu_lora, linear_lora): host-side validation, planning and launches.
#include <algorithm>

#include "api_internal.h"
#include "dense_launch.h"
#include "lora_generic.cuh"
#include "lora_pair.cuh"
#include "lora_shrink_tc.cuh"
#include "pair_plan.h"

namespace {

using namespace mbglu_host;

constexpr int kFewRows = 64;   // a decode batch
constexpr int kJoinRows = 320;

// Who adds the terms of rows with adapters of their own (us at K = 2560, N = 9728, two projections):
//   up to rank 16 the epilogue, a row of B per lane: at 100 rows of as many requests 40, on the
//   tensor cores (lora_term) 59; at 1000 rows of 30 requests 102 and 114, at 4000 248 and 285;
//   of rank 24 the tensor cores up to some 2000 rows and little behind from there (4000 rows of
//   60 requests 330, by rows 322); of rank 64 500 rows of 60 requests 113, by rows 363;
//   a decode batch's larger ranks the join, which has more warps: at 48 rows of rank 64 57, in
//   the epilogue 83; of rank 32 36 and 47.
// With all tiles in the join p needs no kernel of its own: the products hide it.  So smaller ranks
// and larger batches go there too, if the tiles are one round at most (56 column tiles, rank 8:
// 256 rows 55 and 57 us, 300 rows 68 and 61) and forming p takes a block no longer than its
// products (hidden_values): linear, K = 4096, N = 4096, rank 16, joined and not: 8 rows 12.2 and
// 17.9, 64 rows 13.6 and 24.1, 128 rows 17.0 and 30.5; gated, K = 2560, N = 9728: 16 rows 24.3
// and 26.8, 160 rows of rank 32 64 and 70 (of rank 8 43 and 41); gated, K = 1024, N = 2816, 24
// rows, beyond that bound, 12.0 and 11.0.
// Rows and rank end where a chunk of few requests would lose more than a batch of many gains
// (linear, K = 9728, N = 2560, rows of their own and of 4 requests): 160 rows of rank 32 40 and
// 69, 34 and 35; 256 52 and 89, 47 and 37; 333 rows of rank 16 41 and 70, 38 and 37; 510 54 and
// 89, 51 and 44.
bool by_rows(int M, int R) { return M <= kFewRows || R <= 16; }
int64_t hidden_values(int K, int column_tiles) { return static_cast<int64_t>(std::max(K / 512, 1)) * column_tiles * 16; }
bool by_join(int sides, int M, int K, int R, int column_tiles)
{
    const int64_t values = static_cast<int64_t>(M) * sides * R, hidden = hidden_values(K, column_tiles);
    if (M < 2 || values <= mbglu::kInsideMost) return false;
    if (M <= kFewRows && R > 16) return true;
    if (static_cast<int64_t>(column_tiles) * ceil_div(M, mbglu::kPairTile) > kPairs) return false;
    return M <= kFewRows ? values <= hidden : M <= kJoinRows && M * R <= 5120 && values <= 4 * hidden;
}

// A range leaves the sums of a tile's rows, 256 outputs each.
int64_t lora_part_bytes(int64_t ranges, int tn, int M) { return ranges * std::min(tn, M) * 1024; }

// The most ranges that a tile is cut into: 8 chunks each
int64_t most_ranges(int K) { return std::min(std::max(ceil_div(K, 64) / 8, 1), 16); }

// Tiles and ranges, from the sizes and from the room for partial sums alone.  The estimate
// (ns) of a tile's time is tall_tokens' (gemm_api.cu); a join costs its launch, the partial
// sums' way to L2 and back and the adapters' terms (500 x 2560 outputs of R = 32: 24 us).
// Plans of whole tiles need no room.
mbglu::LoraPlan lora_plan(int sides, int M, int N, int K, int R, bool may_split, int64_t room)
{
    mbglu::LoraPlan best = {};
    double least = 0;
    const int chunks = ceil_div(K, 64), wt = sides == 2 ? 128 : 256, nt = ceil_div(N, wt);
    for (int tn = 32; tn <= mbglu::kPairTile; tn += 32) {
        if (tn > 32 && tn - 32 >= M) break;
        const int64_t tiles = static_cast<int64_t>(nt) * ceil_div(M, tn);
        if (tiles > INT32_MAX / 16) continue;
        const auto tile_ns = [&](int64_t at_once, int64_t n) { return n * (77.0 + 59.0 * std::min<int64_t>(at_once, kPairs) / kPairs + 0.7 * tn) + 15.5 * tn; };
        const bool join = may_split && by_join(sides, M, K, R, nt) && lora_part_bytes(tiles, tn, M) <= room;
        for (int split = 0; split < 2; ++split) {
            const int64_t left = join ? tiles : tiles % kPairs;
            const int64_t s = split && left > 0 ? std::min({std::max<int64_t>(kPairs / left, 1), most_ranges(K), room / lora_part_bytes(left, tn, M)}) : 1;
            if (split && !may_split) continue;
            if (join ? !split : split && s < 2) continue;
            const int64_t whole = split ? tiles - left : tiles;
            double ns = (whole + kPairs - 1) / kPairs * tile_ns(whole, chunks);
            if (split) ns += (left * s + kPairs - 1) / kPairs * tile_ns(left * s, (chunks + s - 1) / s) + 3000 + left * s * std::min(tn, M) * 2048.0 / 4000 + left * std::min(tn, M) * 4;
            if (may_split && whole > 0 && M >= 2 && M <= kFewRows && M * sides * R > mbglu::kInsideMost) ns += 4000;   // p's kernel, which nothing hides
            if (least == 0 || ns < least) {
                least = ns;
                best.tn = tn;
                best.wt = wt;
                best.ttiles = ceil_div(M, tn);
                best.ntiles = static_cast<int>(tiles);
                best.whole = static_cast<int>(whole);
                best.rest = split ? static_cast<int>(left) : 0;
                best.splits = static_cast<int>(s);
                best.items = static_cast<int>(whole + (split ? left * s : 0));
                best.nchunk = chunks;
            }
        }
    }
    return best;
}

int64_t lora_p_bytes(int sides, int M, int R) { return padded(static_cast<int64_t>(M) * sides * R * 4); }

// The largest partial sums of any plan of up to M rows: ranges of less than a round of tiles, or
// all tiles of the batches that by_join lets through.
int64_t most_part_bytes(int sides, int M, int N, int K, int R)
{
    const int64_t nt = ceil_div(N, sides == 2 ? 128 : 256);
    const int joined = std::min(M, nt * ceil_div(kJoinRows, mbglu::kPairTile) <= kPairs ? kJoinRows : nt <= kPairs ? mbglu::kPairTile : R > 16 ? kFewRows : 0);
    int64_t most = 0;
    for (int tn = 32; tn <= mbglu::kPairTile && (tn == 32 || tn - 32 < M); tn += 32) {
        most = std::max(most, lora_part_bytes(std::min<int64_t>(kPairs, nt * ceil_div(M, tn) * most_ranges(K)), tn, M));
        if (tn == 32 || tn - 32 < joined) most = std::max(most, lora_part_bytes(nt * ceil_div(joined, tn), tn, joined));
    }
    return most;
}

// From this many rows on p comes from lora_shrink_tc_kernel: at 500 rows of 60 requests, K =
// 9728, the whole call takes 66 us with it and 70 without, at 1000 of 10, K = 2560, 95 and 99;
// at 333 rows of 37 31 and 23.
constexpr int kShrinkTcFrom = 512, kShrinkTcSplit = 8;   // blocks that share a tile
constexpr int kShrinkTcBlocks = 160;                     // and at most in all, where tiles are shared

// Places of the workspace, in bytes: moe_glu's counters, which stay as they are (a decode loop may
// keep one buffer for both), p, its two terms, the table of 32-row blocks, then the partial sums
// of p and of the outputs, one after the other, in what there is behind.
struct LoraSpace {
    int64_t p, terms, blocks, part;
};

LoraSpace lora_space(int sides, int M, int R)
{
    LoraSpace s = {};
    s.p = MBGLU_MOE_COUNTER_BYTES;
    s.terms = s.p + lora_p_bytes(sides, M, R);
    s.blocks = s.terms + lora_p_bytes(sides, M, R);
    s.part = s.blocks + padded((static_cast<int64_t>(M) + mbglu::kLoraBlock - 1) / mbglu::kLoraBlock * 4);
    return s;
}

// Partial sums of p beside the first block's, which lie where p does: of `split` blocks.
int64_t shrink_part_bytes(int sides, int M, int R, int split) { return (split - 1) * static_cast<int64_t>(M) * sides * R * 4; }

// Room for the fastest plan of any number of rows up to M.
int64_t lora_bytes(int sides, int M, int N, int K, int R)
{
    // of more rows fewer blocks share a tile (kShrinkTcBlocks), and their parts are less than these
    const int rows = M < kShrinkTcFrom ? 0 : std::min(M, kShrinkTcBlocks / kShrinkTcSplit * mbglu::kShrinkTcRows);
    return lora_space(sides, M, R).part + padded(std::max(most_part_bytes(sides, M, N, K, R), shrink_part_bytes(sides, rows, R, kShrinkTcSplit)));
}

bool bad_rank(int adapters, int R) { return adapters < 0 || adapters > kMostSize || R < 0 || R > MBGLU_LORA_MAX_RANK; }

// The cluster's blocks split the inner dimension: as many as leave a warp about five steps,
// so that all of its loads are on the way together, and no more than `most` blocks in all.
template <int SIDES, int MT, int NT, int UNROLL>
mbglu_status launch_shrink(const mbglu::LoraParams &p, int side_by_side, int most, cudaStream_t stream)
{
    const int64_t groups = std::min<int64_t>((static_cast<int64_t>(p.M) + MT * 16 - 1) / (MT * 16), 32768);
    const int64_t blocks = groups * SIDES * ceil_div(p.R, NT * 8) * side_by_side;
    int split = 1;
    while (split < 8 && ceil_div(p.K, 32) > 5 * mbglu::kShrinkWarps * split && blocks * split * 2 <= most) split *= 2;
    Launch l(dim3(static_cast<unsigned>(SIDES * ceil_div(p.R, NT * 8) * split), static_cast<unsigned>(groups), static_cast<unsigned>(side_by_side)),
             mbglu::kShrinkWarps * 32, mbglu::shrink_smem<MT, NT>(), stream, split);
    return launched(cudaLaunchKernelEx(&l.cfg, mbglu::lora_shrink_kernel<SIDES, MT, NT, UNROLL>, p, split));
}

// Blocks of a cluster split the inner dimension, so that the tiles of 128 rows fill the SMs.
template <int SIDES>
mbglu_status launch_shrink_tc(const mbglu::LoraParams &p, float *part, int64_t room, bool *taken, cudaStream_t stream)
{
    *taken = false;
    mbglu::ShrinkTcMaps maps;
    if (!encode_tile_map(&maps.x, p.x, p.ldx, p.M, p.K, 64, mbglu::kShrinkTcRows, 2)) return MBGLU_OK;
    for (int d = 0; d < SIDES; ++d) {
        const mbglu::LoraSide &s = p.side[d];
        if ((p.adapters > 1 && s.a_adapter <= 0) || !encode_stack_map(&maps.a[d], s.a, s.a_adapter, s.lda, p.adapters, p.R, p.K, 64, p.R)) return MBGLU_OK;
    }
    const int tiles = ceil_div(p.M, mbglu::kShrinkTcRows);
    if (tiles > 65535) return MBGLU_OK;
    mbglu::ShrinkTcParams q = {};
    q.l = p;
    q.part = part;
    q.nchunk = ceil_div(p.K, 64);
    q.group = mbglu::shrink_tc_group(SIDES * p.R);
    q.split = 1;
    while (q.split < kShrinkTcSplit && tiles * q.split * 2 <= kShrinkTcBlocks && q.nchunk >= q.split * 8 && shrink_part_bytes(SIDES, p.M, p.R, q.split * 2) <= room) q.split *= 2;
    const uint32_t stage = mbglu::shrink_tc_stage(SIDES * p.R);
    q.stages = std::min<int>(mbglu::kShrinkTcMaxStages, (200 * 1024) / static_cast<int>(stage));
    *taken = true;
    Launch l(dim3(static_cast<unsigned>(q.split), static_cast<unsigned>(tiles)), mbglu::kShrinkTcThreads,
             mbglu::kShrinkTcHeader + 1024 + static_cast<size_t>(q.stages) * stage, stream,
             q.split);
    return launched(cudaLaunchKernelEx(&l.cfg, mbglu::lora_shrink_tc_kernel<SIDES>, q, maps));
}

template <int SIDES>
cudaError_t setup_pair()
{
    cudaError_t e = cudaSuccess;
    for (const auto kernel : {mbglu::lora_pair_kernel<SIDES, false>, mbglu::lora_pair_kernel<SIDES, true>})
        if (e == cudaSuccess) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(mbglu::kLoraSmem));
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(mbglu::lora_shrink_tc_kernel<SIDES>, cudaFuncAttributeMaxDynamicSharedMemorySize, 204 * 1024);
    return e;
}

template <int SIDES, int TOKENS, int LANES>
mbglu_status launch_join(const mbglu::LoraPairParams &p, cudaStream_t stream)
{
    const int64_t warps = static_cast<int64_t>(p.plan.rest) * ceil_div(p.plan.wt, 32) * (p.plan.tn / TOKENS);
    Launch j(dim3(static_cast<unsigned>(std::min<int64_t>((warps + 7) / 8, 1 << 20))), 256, 0, stream);
    return launched(cudaLaunchKernelEx(&j.cfg, mbglu::lora_join_kernel<SIDES, TOKENS, LANES>, p));
}

template <int SIDES>
mbglu_status launch_join(const mbglu::LoraPairParams &p, cudaStream_t stream)
{
    const int R = p.l.R;
    if (p.l.M <= 16) {   // more warps, each with less
        if (R <= 16) return launch_join<SIDES, 1, 2>(p, stream);
        if (R <= 32) return launch_join<SIDES, 1, 4>(p, stream);
    } else {
        if (R <= 16) return launch_join<SIDES, 2, 2>(p, stream);
        if (R <= 32) return launch_join<SIDES, 2, 4>(p, stream);
    }
    if (R <= 64) return launch_join<SIDES, 1, 8>(p, stream);
    return launch_join<SIDES, 1, 16>(p, stream);
}

// Operands that the CTA-pair kernel and lora_shrink_kernel take.
bool fast_operands(const mbglu::LoraParams &p, int sides)
{
    if (p.K == 0 || !copyable(p.x, p.ldx, 2)) return false;
    for (int d = 0; d < sides; ++d) {
        const mbglu::LoraSide &s = p.side[d];
        if (!copyable(s.w, s.ldw, 2)) return false;
        if (p.adapters == 0) continue;
        // rows are read 16 bytes at a time, the last ones too
        if (p.K % 8 != 0 || p.R % 8 != 0 || !copyable(s.a, s.lda, 2) || !copyable(s.b, s.ldb, 2)) return false;
        if (p.adapters > 1 && (s.a_adapter % 8 != 0 || s.b_adapter % 8 != 0)) return false;
    }
    return true;
}

template <int SIDES>
mbglu_status launch_pair(const mbglu::LoraParams &l, const mbglu::LoraPlan &plan, void *workspace, const LoraSpace &space, int64_t room, bool *taken,
                         cudaStream_t stream)
{
    *taken = false;
    if (!fast_operands(l, SIDES) || plan.ntiles == 0) return MBGLU_OK;
    mbglu::LoraPairParams p = {};
    p.l = l;
    p.plan = plan;
    p.rows = std::min(plan.tn, l.M);
    char *ws = static_cast<char *>(workspace);
    const bool adapted = l.adapters > 0, whole = p.plan.whole > 0;
    mbglu::LoraMaps maps;
    for (int d = 0; d < SIDES; ++d)
        if (!encode_tile_map(&maps.w[d], l.side[d].w, l.side[d].ldw, l.N, l.K, 64, p.plan.wt / 2, 2)) return MBGLU_OK;
    if (!encode_tile_map(&maps.x, l.x, l.ldx, l.M, l.K, 64, p.plan.tn / 2, 2)) return MBGLU_OK;
    if (adapted) {
        const int width = SIDES * l.R;
        // 10 MB of B or less (48 rows of rank 32, 60 MB: 40 us with and 36 without; of rank 16 31.5
        // and 30.7)
        p.prefetch = static_cast<int64_t>(std::min(l.M, l.adapters)) * l.N * width * 2 <= 10000000;
        // p is formed beside the products of a plan without whole tiles where that takes no longer
        // than a kernel of its own: 64 rows of rank 64, K = 2560, N = 9728 62 us and 70; K = 1024, N =
        // 2816, beyond the bound, 40 and 33
        const int column_tiles = ceil_div(l.N, p.plan.wt);
        if (!whole && (l.M <= kFewRows ? static_cast<int64_t>(l.M) * width <= 4 * hidden_values(l.K, column_tiles)
                                       : by_join(SIDES, l.M, l.K, l.R, column_tiles)))
            p.inside = mbglu::kInsideShared;
        else if (by_rows(l.M, l.R) && p.plan.rest == 0 && static_cast<int64_t>(l.M) * width <= mbglu::kInsideMost)
            p.inside = mbglu::kInsideEach;
        p.l.terms = reinterpret_cast<uint16_t *>(ws + space.terms);
        p.part = reinterpret_cast<float *>(ws + space.part);
        if (whole && p.inside == mbglu::kInsideNo) {   // tiles in ranges leave the adapters' term to the join
            p.l.blocks = reinterpret_cast<int32_t *>(ws + space.blocks);
            for (int d = 0; d < SIDES; ++d) {
                const mbglu::LoraSide &s = l.side[d];
                if ((l.adapters > 1 && s.b_adapter <= 0) ||
                    !encode_stack_map(&maps.b[d], s.b, s.b_adapter, s.ldb, l.adapters, l.N, l.R, 64, p.plan.wt / 2))
                    return MBGLU_OK;
            }
            for (int i = 0; i < 2; ++i)
                if (!encode_tile_map(&maps.p[i], p.l.terms + static_cast<int64_t>(i) * l.M * width, width, l.M, width, 64, 16, 2)) return MBGLU_OK;
        }
    }
    static DeviceTable table;
    int sms = 0;
    mbglu_status st = table.get(&sms, setup_pair<SIDES>);
    if (st != MBGLU_OK) return st;
    *taken = true;
    if (adapted && p.inside == mbglu::kInsideNo) {
        // few rows: a block per adapter of a group and 8 columns; many: columns together, so
        // that the rows are read once or twice
        p.early = launch_policy() != MBGLU_POLICY_SERIAL;
        bool tc = false;
        if (l.M >= kShrinkTcFrom) st = launch_shrink_tc<SIDES>(p.l, p.part, room, &tc, stream);
        if (st == MBGLU_OK && !tc) {
            if (l.M <= kFewRows)
                st = launch_shrink<SIDES, 1, 1, 5>(p.l, std::min(l.M, 16), 1024, stream);
            else   // blocks without an adapter of theirs leave at once
                st = launch_shrink<SIDES, 1, 4, 4>(p.l, 8, 608, stream);
        }
        if (st != MBGLU_OK) return st;
    }
    p.ahead = !p.early && launch_policy() == MBGLU_POLICY_PREFETCH;
    Launch c(dim3(static_cast<unsigned>(2 * std::min(std::max(sms / 2, 1), p.plan.items))), mbglu::kPairThreads, mbglu::kLoraSmem, stream, 2);
    const auto kernel = by_rows(l.M, l.R) || p.inside != mbglu::kInsideNo ? mbglu::lora_pair_kernel<SIDES, true> : mbglu::lora_pair_kernel<SIDES, false>;
    st = launched(cudaLaunchKernelEx(&c.cfg, kernel, p, maps));
    if (st == MBGLU_OK && p.plan.rest > 0) st = launch_join<SIDES>(p, stream);
    return st;
}

template <int SIDES>
mbglu_status run(mbglu::LoraParams &p, void *workspace, size_t workspace_bytes, cudaStream_t stream)
{
    const int M = p.M, N = p.N, K = p.K, R = p.R;
    if (p.mode != MBGLU_MODE_FUSED && p.mode != MBGLU_MODE_HF) return MBGLU_ERR_MODE;
    if (bad_sizes(M, N, K) || N > INT32_MAX / 2 || bad_rank(p.adapters, R)) return MBGLU_ERR_SHAPE;
    if (M == 0 || N == 0) return MBGLU_OK;
    if (R == 0 || K == 0) p.adapters = 0;   // the second term is an empty sum
    const bool adapted = p.adapters > 0;
    if (!p.out || (K > 0 && !p.x) || (adapted && (!p.adapter || !workspace))) return MBGLU_ERR_NULL;
    for (int d = 0; d < SIDES; ++d)
        if ((K > 0 && !p.side[d].w) || (adapted && (!p.side[d].a || !p.side[d].b))) return MBGLU_ERR_NULL;
    if (p.ldo < N || (K > 0 && p.ldx < K)) return MBGLU_ERR_STRIDE;
    for (int d = 0; d < SIDES; ++d) {
        const mbglu::LoraSide &s = p.side[d];
        if (K > 0 && s.ldw < K) return MBGLU_ERR_STRIDE;
        if (adapted && (s.lda < K || s.ldb < R || (p.adapters > 1 && (s.a_adapter < 0 || s.b_adapter < 0)))) return MBGLU_ERR_STRIDE;
    }
    bool ok = aligned(p.out, 2) && aligned(p.x, 2);
    for (int d = 0; d < SIDES; ++d) ok = ok && aligned(p.side[d].w, 2);
    if (adapted) {
        ok = ok && aligned(p.adapter, 4) && aligned(p.scale, 4) && aligned(workspace, kAlign);
        for (int d = 0; d < SIDES; ++d) ok = ok && aligned(p.side[d].a, 2) && aligned(p.side[d].b, 2);
    }
    if (!ok) return MBGLU_ERR_ALIGN;
    // p and its table have to fit; partial sums get what is left, up to what they can use
    const LoraSpace space = lora_space(SIDES, M, R);
    const int64_t has = adapted ? std::min<int64_t>(std::min<size_t>(workspace_bytes, INT64_MAX), lora_bytes(SIDES, M, N, K, R)) : 0;
    if (adapted && has < space.part) return MBGLU_ERR_SHAPE;
    const void *outs[2] = {p.out, workspace};
    const int64_t outb[2] = {extent(M, N, p.ldo, 2), has};
    if (overlaps(outs[0], outb[0], outs[1], outb[1])) return MBGLU_ERR_ALIAS;
    for (int i = 0; i < 2; ++i) {
        if (overlaps(outs[i], outb[i], p.x, extent(M, K, p.ldx, 2))) return MBGLU_ERR_ALIAS;
        for (int d = 0; d < SIDES; ++d) {
            const mbglu::LoraSide &s = p.side[d];
            if (overlaps(outs[i], outb[i], s.w, extent(N, K, s.ldw, 2))) return MBGLU_ERR_ALIAS;
            if (adapted && (overlaps(outs[i], outb[i], s.a, extent3(p.adapters, R, K, s.a_adapter, s.lda)) ||
                            overlaps(outs[i], outb[i], s.b, extent3(p.adapters, N, R, s.b_adapter, s.ldb))))
                return MBGLU_ERR_ALIAS;
        }
        if (adapted && (overlaps(outs[i], outb[i], p.adapter, static_cast<int64_t>(M) * 4) ||
                        overlaps(outs[i], outb[i], p.scale, p.scale ? static_cast<int64_t>(p.adapters) * 4 : 0)))
            return MBGLU_ERR_ALIAS;
    }
    p.p = adapted ? reinterpret_cast<float *>(static_cast<char *>(workspace) + space.p) : nullptr;   // the kernels for any alignment need no more
    bool taken = false;
    const int64_t room = adapted ? has - space.part : 0;
    mbglu_status st = launch_pair<SIDES>(p, lora_plan(SIDES, M, N, K, R, adapted, room), workspace, space, room, &taken, stream);
    if (taken || st != MBGLU_OK) {
        if (st == MBGLU_OK) set_last_variant(kLoraPair);
        return st;
    }
    if (adapted) {
        const int64_t warps = static_cast<int64_t>(M) * SIDES * R;
        Launch l(dim3(static_cast<unsigned>(std::min<int64_t>((warps + 7) / 8, 1 << 20))), 256, 0, stream);
        st = launched(cudaLaunchKernelEx(&l.cfg, mbglu::lora_generic_shrink<SIDES>, p));
    }
    if (st == MBGLU_OK) {
        Launch l(mbglu::gen_grid(M, N), 256, 0, stream);
        st = launched(cudaLaunchKernelEx(&l.cfg, mbglu::lora_generic_kernel<SIDES>, p));
    }
    if (st == MBGLU_OK) set_last_variant(kLoraGeneric);
    return st;
}

mbglu::LoraSide side(const mbglu_bf16 *w, int64_t ldw, const mbglu_adapters *q)
{
    mbglu::LoraSide s = {};
    s.w = w;
    s.ldw = ldw;
    if (q) {
        s.a = q->a;
        s.a_adapter = q->a_adapter;
        s.lda = q->lda;
        s.b = q->b;
        s.b_adapter = q->b_adapter;
        s.ldb = q->ldb;
    }
    return s;
}

mbglu::LoraParams params(const mbglu_bf16 *x, int64_t ldx, const int32_t *adapter, const float *scale, mbglu_bf16 *out, int64_t ldo,
                         int M, int N, int K, int adapters, int R, int mode)
{
    mbglu::LoraParams p = {};
    p.x = x;
    p.ldx = ldx;
    p.adapter = adapter;
    p.scale = scale;
    p.out = out;
    p.ldo = ldo;
    p.M = M;
    p.N = N;
    p.K = K;
    p.adapters = adapters;
    p.R = R;
    p.mode = mode;
    return p;
}

}  // namespace

extern "C" {

size_t glu_lora_workspace_bytes(int M, int N, int K, int adapters, int R)
{
    if (bad_sizes(M, N, K) || N > INT32_MAX / 2 || bad_rank(adapters, R) || std::min({M, N, K, adapters, R}) == 0) return 0;
    return static_cast<size_t>(lora_bytes(2, M, N, K, R));
}

size_t linear_lora_workspace_bytes(int M, int N, int K, int adapters, int R)
{
    if (bad_sizes(M, N, K) || N > INT32_MAX / 2 || bad_rank(adapters, R) || std::min({M, N, K, adapters, R}) == 0) return 0;
    return static_cast<size_t>(lora_bytes(1, M, N, K, R));
}

mbglu_status glu_lora(const mbglu_bf16 *h, int64_t ldh, const mbglu_bf16 *gate_w, int64_t ld_gate, const mbglu_bf16 *up_w, int64_t ld_up,
                      const mbglu_adapters *gate, const mbglu_adapters *up, const int32_t *adapter, const float *scale,
                      mbglu_bf16 *out, int64_t ldo, int M, int N, int K, int adapters, int R, mbglu_mode mode,
                      void *workspace, size_t workspace_bytes, cudaStream_t stream)
{
    set_last_variant(0);
    mbglu::LoraParams p = params(h, ldh, adapter, scale, out, ldo, M, N, K, adapters, R, static_cast<int>(mode));
    p.side[0] = side(gate_w, ld_gate, gate);
    p.side[1] = side(up_w, ld_up, up);
    return run<2>(p, workspace, workspace_bytes, stream);
}

mbglu_status linear_lora(const mbglu_bf16 *x, int64_t ldx, const mbglu_bf16 *w, int64_t ldw, const mbglu_adapters *ab,
                         const int32_t *adapter, const float *scale, mbglu_bf16 *out, int64_t ldo,
                         int M, int N, int K, int adapters, int R, void *workspace, size_t workspace_bytes, cudaStream_t stream)
{
    set_last_variant(0);
    mbglu::LoraParams p = params(x, ldx, adapter, scale, out, ldo, M, N, K, adapters, R, MBGLU_MODE_FUSED);
    p.side[0] = side(w, ldw, ab);
    return run<1>(p, workspace, workspace_bytes, stream);
}

}  // extern "C"

namespace mbglu_host {

cudaError_t take_lora_error(int *w)
{
    cudaError_t e = cudaMemcpyFromSymbol(w, mbglu::g_dense_error, sizeof *w);
    const int zero = 0;
    return e != cudaSuccess ? e : cudaMemcpyToSymbol(mbglu::g_dense_error, &zero, sizeof zero);
}

}  // namespace mbglu_host
