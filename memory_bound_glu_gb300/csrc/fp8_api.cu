// fp8_api.cu -- the gated block with e4m3 operands and block scales
// (add_rmsnorm_fp8, glu_fp8, matmul_fp8, quantize_weight_fp8): host-side
// validation, planning and launches.
#include <algorithm>

#include "api_internal.h"
#include "dense_generic.cuh"
#include "dense_launch.h"
#include "fp8_pair.cuh"
#include "fp8_tall.cuh"
#include "norm_fp8.cuh"
#include "pair_plan.h"

namespace {

using namespace mbglu_host;

constexpr int64_t kBlk = mbglu::kScaleBlock;

mbglu::GenOperand operand(const uint8_t *p, int64_t ld, const float *scale, int64_t lds)
{
    return mbglu::GenOperand{p, ld, 1, scale, lds};
}

template <int EPI, bool DUAL>
mbglu_status launch_generic(const mbglu::GenParams &p, cudaStream_t stream)
{
    Launch l(mbglu::gen_grid(p.rows, p.cols), 256, 0, stream);
    const mbglu_status st = launched(cudaLaunchKernelEx(&l.cfg, mbglu::dense_generic_kernel<EPI, true, DUAL>, p));
    if (st == MBGLU_OK) set_last_variant(kFp8Generic);
    return st;
}

// One e4m3 operand with its scales: [rows][K], scales [scale_rows][blocks of K]
struct Scaled {
    const uint8_t *p;
    int64_t ld;
    const float *s;
    int64_t lds;
    int64_t rows, scale_rows;
};

mbglu_status check_scaled(const Scaled &o, int K)
{
    if (K == 0) return MBGLU_OK;
    if (!o.p || !o.s) return MBGLU_ERR_NULL;
    if (o.ld < K || o.lds < ceil_div(K, kBlk)) return MBGLU_ERR_STRIDE;
    return aligned(o.s, 4) ? MBGLU_OK : MBGLU_ERR_ALIGN;
}

bool meets(const void *p, int64_t bytes, const Scaled &o, int K)
{
    return K > 0 && (overlaps(p, bytes, o.p, extent(o.rows, K, o.ld, 1)) ||
                     overlaps(p, bytes, o.s, extent(o.scale_rows, ceil_div(K, kBlk), o.lds, 4)));
}

template <int EPI>
cudaError_t allow_pair()
{
    return cudaFuncSetAttribute(mbglu::fp8_pair_kernel<EPI>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                static_cast<int>(mbglu::kFp8Smem));
}

cudaError_t setup_tall();

cudaError_t setup_fp8()
{
    cudaError_t e = allow_pair<mbglu::kFp8Out>();
    if (e == cudaSuccess) e = allow_pair<mbglu::kFp8Glu>();
    if (e == cudaSuccess) e = allow_pair<mbglu::kFp8GluQuant>();
    if (e == cudaSuccess) e = setup_tall();
    return e;
}

mbglu_status sm_count(int *n)
{
    static DeviceTable table;
    return table.get(n, setup_fp8);
}

// A map of 128 columns x box_rows; false where tensor copies do not take the
// operand.  The stride of a single row is never used: any multiple of 16 does.
bool k_major(mbglu::TensorMap *m, const Scaled &o, int K, int box_rows = 128)
{
    const int64_t ld = o.rows == 1 ? (o.ld + 15) / 16 * 16 : o.ld;
    return copyable(o.p, ld, 1) && encode_tile_map(m, o.p, ld, static_cast<int>(o.rows), K, 128, box_rows, 1);
}

template <int EPI>
mbglu_status launch_pair(const mbglu::Fp8PairParams &p, const mbglu::PairMaps &maps, cudaStream_t stream)
{
    int sms = 0;
    mbglu_status st = sm_count(&sms);
    if (st != MBGLU_OK) return st;
    Launch l(dim3(static_cast<unsigned>(2 * std::min(std::max(sms / 2, 1), p.plan.ntiles))), mbglu::kPairThreads, mbglu::kFp8Smem,
             stream, 2);
    st = launched(cudaLaunchKernelEx(&l.cfg, mbglu::fp8_pair_kernel<EPI>, p, maps));
    if (st == MBGLU_OK) set_last_variant(kFp8Pair);
    return st;
}

// ---- few rows, or few tiles: fp8_tall_kernel ----------------------------------------------

// Clusters of ks blocks, each with an SM of its own, that the part holds at once
// (tall_per_sm: some have two per SM).
constexpr int kClusters[mbglu::kTallMaxSplit + 1] = {0, 152, 76, 46, 36, 28, 23, 15, 15};

constexpr int kTallTokens[] = {16, 32, 48, 64, 80, 96, 112, 128};   // two weights: up to 48

// Which kernel, tokens per block (tn) and ranges of the inner dimension (ks): what
// makes the estimate of a call's time in a chain of calls least.  From the sizes
// alone, so that the order of a sum does not depend on the device.  The constants
// (ns) are fitted to 2,500 measured combinations of tn and ks, 16 to 768 rows, six
// shapes of one weight and five of two.  There the choice is within 1% of the fastest
// combination on average and 10% at worst, and so it is at eleven other shapes of 333
// to 4096 rows.  It is faster by 20% (one weight) and 17% (two) on average than the
// least tn that holds all rows, up to 128 (two weights: 64), and CTA pairs beyond; slower
// by 2% or more at three points: two weights of K = 4096, N = 11008 and 48 and 64 rows
// (26.6 and 30.2 us against 26.0 and 28.1), K = 2048, N = 4096 and 16 rows (7.2 and 6.8).
struct TallCost {
    int64_t start, stage, stage_col, col, round, paired, rank, block;
};
struct PairCost {
    int64_t start, stage, stage_full, join, join_slot;
};
constexpr TallCost kTallCost[2] = {{500, 210, 1, 50, 300, 350, 75, 1100}, {1000, 290, 2, 57, 0, 2500, 276, 820}};
constexpr PairCost kPairCost[2] = {{5300, 360, 130, 1800, 95}, {6600, 330, 160, 0, 0}};

struct TallPlan {
    int tn, ks;
    int64_t ns;
};

TallPlan tall_plan(int M, int N, int K, bool dual)
{
    const TallCost &c = kTallCost[dual];
    const int64_t wtiles = ceil_div(N, mbglu::kTallRows);
    const int chunks = ceil_div(K, kBlk);
    TallPlan t = {};
    for (const int tn : kTallTokens) {
        if (dual && tn > 48) break;   // would hardly ever be the least
        const int64_t units = wtiles * ceil_div(M, tn), cols = (dual ? 2 : 1) * tn;
        const int per_sm = mbglu::tall_per_sm(tn, dual);
        for (int ks = 1; ks <= std::min(mbglu::kTallMaxSplit, chunks); ++ks) {
            const int places = kClusters[ks] * per_sm;
            const int64_t round = ceil_div(chunks, ks) * (c.stage + c.stage_col * cols) + c.col * cols + c.round +
                                  (per_sm == 2 ? c.paired : 0);
            const int64_t ns = c.start + (units + places - 1) / places * round + c.rank * ks + c.block * units * ks / (2 * kPairs);
            if (t.tn == 0 || ns < t.ns) t = {tn, ks, ns};
        }
        if (tn >= M) break;   // wider tiles would only be emptier
    }
    return t;
}

int64_t pair_ns(const mbglu::PairPlan &p, bool dual)
{
    const PairCost &c = kPairCost[dual];
    const int64_t stages = static_cast<int64_t>(ceil_div(p.whole, kPairs)) * p.nchunk + (p.rest ? ceil_div(p.nchunk, p.splits) : 0);
    return c.start + stages * (c.stage + c.stage_full * std::min(p.ntiles, kPairs) / kPairs) +
           (p.rest ? c.join + c.join_slot * p.rest * p.splits : 0);
}

// One weight: every stage is of a[0] and b[0], the only maps that are filled in.
mbglu::PairPlan fp8_pair_plan(int M, int N, int K, bool dual, bool may_split)
{
    const int chunks = ceil_div(K, kBlk);
    return pair_plan(M, N, dual ? 128 : 256, 1, chunks, chunks, may_split);
}

struct Fp8Plan {
    TallPlan tall;
    mbglu::PairPlan pair;
    bool use_tall;
};

Fp8Plan fp8_plan(int M, int N, int K, bool dual)
{
    Fp8Plan f = {};
    f.pair = fp8_pair_plan(M, N, K, dual, !dual);
    if (K > 0) {
        f.tall = tall_plan(M, N, K, dual);
        f.use_tall = f.tall.ns < pair_ns(f.pair, dual);
    }
    return f;
}

template <int TN, int OUT>
cudaError_t allow_tall()
{
    return cudaFuncSetAttribute(mbglu::fp8_tall_kernel<TN, OUT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                static_cast<int>(mbglu::TallShape<TN, OUT != 0>::kSmem));
}

cudaError_t setup_tall()
{
    cudaError_t e = cudaSuccess;
#define MBGLU_ALLOW(TN, OUT) \
    if (e == cudaSuccess) e = allow_tall<TN, OUT>();
    MBGLU_ALLOW(16, 0) MBGLU_ALLOW(32, 0) MBGLU_ALLOW(48, 0) MBGLU_ALLOW(64, 0)
    MBGLU_ALLOW(80, 0) MBGLU_ALLOW(96, 0) MBGLU_ALLOW(112, 0) MBGLU_ALLOW(128, 0)
    MBGLU_ALLOW(16, 1) MBGLU_ALLOW(32, 1) MBGLU_ALLOW(48, 1)
    MBGLU_ALLOW(16, 2) MBGLU_ALLOW(32, 2) MBGLU_ALLOW(48, 2)
#undef MBGLU_ALLOW
    return e;
}

template <int TN, int OUT>
mbglu_status launch_tall(const TallPlan &t, const mbglu::TallParams &p, const mbglu::TallMaps &maps, cudaStream_t stream)
{
    const int64_t blocks = static_cast<int64_t>(p.wtiles) * ceil_div(p.M, TN) * t.ks;
    Launch l(dim3(static_cast<unsigned>(blocks)), 384, mbglu::TallShape<TN, OUT != 0>::kSmem, stream, t.ks);
    const mbglu_status st = launched(cudaLaunchKernelEx(&l.cfg, mbglu::fp8_tall_kernel<TN, OUT>, p, maps));
    if (st == MBGLU_OK) set_last_variant(kFp8Tall);
    return st;
}

// False where a tensor map is refused (nothing is launched).
template <int OUT>
bool tall(const TallPlan &t, const Scaled &a, const Scaled &w0, const Scaled *w1, mbglu::TallParams &p, int M, int N, int K,
          cudaStream_t stream, mbglu_status *st)
{
    mbglu::TallMaps maps;
    if (!k_major(&maps.w[0], w0, K) || (w1 && !k_major(&maps.w[1], *w1, K)) || !k_major(&maps.x, a, K, t.tn))
        return false;
    int sms = 0;
    if ((*st = sm_count(&sms)) != MBGLU_OK) return true;
    p.M = M;
    p.N = N;
    p.nchunk = ceil_div(K, kBlk);
    p.ks = t.ks;
    p.wtiles = ceil_div(N, mbglu::kTallRows);
    p.prefetch = launch_policy() == MBGLU_POLICY_PREFETCH;
    p.as = a.s;
    p.ldas = a.lds;
    p.ws[0] = w0.s;
    p.ldws[0] = w0.lds;
    if (w1) {
        p.ws[1] = w1->s;
        p.ldws[1] = w1->lds;
    }
    if constexpr (OUT == 0) {
        if (t.tn > 48) {
            *st = t.tn == 64    ? launch_tall<64, OUT>(t, p, maps, stream)
                  : t.tn == 80  ? launch_tall<80, OUT>(t, p, maps, stream)
                  : t.tn == 96  ? launch_tall<96, OUT>(t, p, maps, stream)
                  : t.tn == 112 ? launch_tall<112, OUT>(t, p, maps, stream)
                                : launch_tall<128, OUT>(t, p, maps, stream);
            return true;
        }
    }
    *st = t.tn == 16   ? launch_tall<16, OUT>(t, p, maps, stream)
          : t.tn == 32 ? launch_tall<32, OUT>(t, p, maps, stream)
                       : launch_tall<48, OUT>(t, p, maps, stream);
    return true;
}

size_t workspace_of(const Fp8Plan &f) { return f.use_tall ? 0 : static_cast<size_t>(part_bytes(f.pair)); }

}  // namespace

extern "C" {

mbglu_status add_rmsnorm_fp8(const mbglu_bf16 *x, int64_t ldx, const mbglu_bf16 *residual, int64_t ldr,
                             mbglu_bf16 *residual_out, int64_t ldro, const mbglu_bf16 *norm_w, float eps, uint8_t *q,
                             int64_t ldq, float *scale, int64_t lds, int M, int K, cudaStream_t stream)
{
    set_last_variant(0);
    if (bad_sizes(M, K) || K < 1) return MBGLU_ERR_SHAPE;
    if (M == 0) return MBGLU_OK;
    if (!x || !residual || !residual_out || !norm_w || !q || !scale) return MBGLU_ERR_NULL;
    if (ldx < K || ldr < K || ldro < K || ldq < K || lds < ceil_div(K, kBlk)) return MBGLU_ERR_STRIDE;
    if (!aligned(x, 2) || !aligned(residual, 2) || !aligned(residual_out, 2) || !aligned(norm_w, 2) ||
        !aligned(scale, 4))
        return MBGLU_ERR_ALIGN;
    const void *ins[3] = {x, residual, norm_w};
    const int64_t ldi[3] = {ldx, ldr, K};
    const int64_t inb[3] = {extent(M, K, ldx, 2), extent(M, K, ldr, 2), extent(1, K, K, 2)};
    const void *outs[3] = {residual_out, q, scale};
    const int64_t outb[3] = {extent(M, K, ldro, 2), extent(M, K, ldq, 1), extent(M, ceil_div(K, kBlk), lds, 4)};
    for (int i = 0; i < 3; ++i) {
        for (int j = 0; j < 3; ++j) {
            // in place: residual_out may be x or residual itself, element by element
            if (i == 0 && j < 2 && outs[0] == ins[j] && (ldro == ldi[j] || M == 1)) continue;
            if (overlaps(outs[i], outb[i], ins[j], inb[j])) return MBGLU_ERR_ALIAS;
        }
        for (int j = i + 1; j < 3; ++j)
            if (overlaps(outs[i], outb[i], outs[j], outb[j])) return MBGLU_ERR_ALIAS;
    }
    mbglu::NormFp8Params p = {x, ldx, residual, ldr, residual_out, ldro, norm_w, eps, q, ldq, scale, lds, M, K};
    // in registers up to 16384 columns; a row's threads: a multiple of a warp, the
    // fewest that leave a thread at most one, two, four or eight chunks of 8
    // columns.  The same for the kernel of any alignment, which then sums in the
    // same order.
    const bool vec = K % 8 == 0 && K <= 16384 && aligned(x, 16) && aligned(residual, 16) && aligned(residual_out, 16) &&
                     aligned(norm_w, 16) && aligned(q, 8) && ldx % 8 == 0 && ldr % 8 == 0 && ldro % 8 == 0 && ldq % 8 == 0;
    const int chunks = ceil_div(K, 8), ch = chunks <= 256 ? 1 : chunks <= 512 ? 2 : chunks <= 1024 ? 4 : 8;
    const int threads = std::min(256, ceil_div(ceil_div(chunks, ch), 32) * 32);
    Launch l(dim3(static_cast<unsigned>(M)), threads, 0, stream);
    const mbglu_status st = launched(!vec      ? cudaLaunchKernelEx(&l.cfg, mbglu::norm_fp8_any_kernel, p)
                                     : ch == 1 ? cudaLaunchKernelEx(&l.cfg, mbglu::norm_fp8_kernel<1>, p)
                                     : ch == 2 ? cudaLaunchKernelEx(&l.cfg, mbglu::norm_fp8_kernel<2>, p)
                                     : ch == 4 ? cudaLaunchKernelEx(&l.cfg, mbglu::norm_fp8_kernel<4>, p)
                                               : cudaLaunchKernelEx(&l.cfg, mbglu::norm_fp8_kernel<8>, p));
    if (st == MBGLU_OK) set_last_variant(kNormFp8);
    return st;
}

mbglu_status quantize_weight_fp8(const mbglu_bf16 *w, int64_t ldw, uint8_t *q, int64_t ldq, float *scale, int64_t lds,
                                 int N, int K, cudaStream_t stream)
{
    set_last_variant(0);
    if (bad_sizes(N, K)) return MBGLU_ERR_SHAPE;
    if (N == 0 || K == 0) return MBGLU_OK;
    if (!w || !q || !scale) return MBGLU_ERR_NULL;
    if (ldw < K || ldq < K || lds < ceil_div(K, kBlk)) return MBGLU_ERR_STRIDE;
    if (!aligned(w, 2) || !aligned(scale, 4)) return MBGLU_ERR_ALIGN;
    const int64_t wb = extent(N, K, ldw, 2), qb = extent(N, K, ldq, 1);
    const int64_t sb = extent(ceil_div(N, kBlk), ceil_div(K, kBlk), lds, 4);
    if (overlaps(q, qb, w, wb) || overlaps(scale, sb, w, wb) || overlaps(q, qb, scale, sb)) return MBGLU_ERR_ALIAS;
    const int nb = ceil_div(N, kBlk);
    Launch l(dim3(static_cast<unsigned>(ceil_div(K, kBlk)), static_cast<unsigned>(std::min(nb, 32768))), 256, 0, stream);
    const mbglu_status st = launched(cudaLaunchKernelEx(&l.cfg, mbglu::quant_weight_kernel, static_cast<const uint16_t *>(w),
                                                        ldw, q, ldq, scale, lds, N, K));
    if (st == MBGLU_OK) set_last_variant(kQuantWeight);
    return st;
}

size_t matmul_fp8_workspace_bytes(int M, int N, int K)
{
    if (M <= 0 || N <= 0 || K <= 0 || bad_sizes(M, N, K)) return 0;
    return workspace_of(fp8_plan(M, N, K, false));
}

mbglu_status matmul_fp8(const uint8_t *a, int64_t lda, const float *a_scale, int64_t ldas, const uint8_t *w,
                        int64_t ldw, const float *w_scale, int64_t ldws, mbglu_bf16 *out, int64_t ldo, int M, int N,
                        int K, void *workspace, size_t workspace_bytes, cudaStream_t stream)
{
    set_last_variant(0);
    if (bad_sizes(M, N, K)) return MBGLU_ERR_SHAPE;
    if (M == 0 || N == 0) return MBGLU_OK;
    if (!out) return MBGLU_ERR_NULL;
    const Scaled A = {a, lda, a_scale, ldas, M, M}, W = {w, ldw, w_scale, ldws, N, ceil_div(N, kBlk)};
    for (const Scaled *o : {&A, &W}) {
        const mbglu_status st = check_scaled(*o, K);
        if (st != MBGLU_OK) return st;
    }
    if (ldo < N) return MBGLU_ERR_STRIDE;
    if (!aligned(out, 2)) return MBGLU_ERR_ALIGN;
    const Fp8Plan plan = fp8_plan(M, N, K, false);
    const size_t need = workspace_of(plan);
    if (need && !workspace) return MBGLU_ERR_NULL;
    if (workspace_bytes < need) return MBGLU_ERR_SHAPE;
    if (need && !aligned(workspace, 256)) return MBGLU_ERR_ALIGN;
    const int64_t ob = extent(M, N, ldo, 2), wsb = static_cast<int64_t>(need);
    if (meets(out, ob, A, K) || meets(out, ob, W, K) || meets(workspace, wsb, A, K) || meets(workspace, wsb, W, K) ||
        overlaps(out, ob, workspace, wsb))
        return MBGLU_ERR_ALIAS;
    if (plan.use_tall) {
        mbglu::TallParams q = {};
        q.out = out;
        q.ldo = ldo;
        mbglu_status st;
        if (tall<0>(plan.tall, A, W, nullptr, q, M, N, K, stream, &st)) return st;
    }
    mbglu::PairMaps maps;
    if (K > 0 && k_major(&maps.a[0], A, K) && k_major(&maps.b[0], W, K)) {
        mbglu::Fp8PairParams q = {};
        q.plan = plan.pair;
        if (plan.use_tall) q.plan = fp8_pair_plan(M, N, K, false, false);   // there is no workspace
        q.as = a_scale;
        q.ldas = ldas;
        q.ws[0] = w_scale;
        q.ldws[0] = ldws;
        q.wblocks = ceil_div(N, kBlk);
        q.out = out;
        q.ldo = ldo;
        q.out_align = row_align(out, ldo, 2);
        q.part = static_cast<float *>(workspace);
        const mbglu_status st = launch_pair<mbglu::kFp8Out>(q, maps, stream);
        uint16_t *const outs[2] = {out, nullptr};
        const int64_t ldos[2] = {ldo, 0};
        return st == MBGLU_OK ? launch_join(q.plan, q.part, outs, ldos, stream) : st;
    }
    mbglu::GenParams p = {};
    p.a[0] = operand(a, lda, a_scale, ldas);
    p.b[0] = operand(w, ldw, w_scale, ldws);
    p.rows = M;
    p.cols = N;
    p.T = K;
    p.npair = 1;
    p.out = out;
    p.ldo = ldo;
    return launch_generic<mbglu::kGenPlain, false>(p, stream);
}

mbglu_status glu_fp8(const uint8_t *a, int64_t lda, const float *a_scale, int64_t ldas, const uint8_t *gate_w,
                     int64_t ld_gate, const float *gate_scale, int64_t ldgs, const uint8_t *up_w, int64_t ld_up,
                     const float *up_scale, int64_t ldus, mbglu_bf16 *out, int64_t ldo, uint8_t *q, int64_t ldq,
                     float *q_scale, int64_t ldqs, int M, int N, int K, cudaStream_t stream)
{
    set_last_variant(0);
    if (bad_sizes(M, N, K)) return MBGLU_ERR_SHAPE;
    if (M == 0 || N == 0) return MBGLU_OK;
    // one form of the output: bf16, or e4m3 with its scales
    if ((out != nullptr) == (q != nullptr) || (q != nullptr) != (q_scale != nullptr)) return MBGLU_ERR_NULL;
    const Scaled A = {a, lda, a_scale, ldas, M, M}, G = {gate_w, ld_gate, gate_scale, ldgs, N, ceil_div(N, kBlk)},
                 U = {up_w, ld_up, up_scale, ldus, N, ceil_div(N, kBlk)};
    for (const Scaled *o : {&A, &G, &U}) {
        const mbglu_status st = check_scaled(*o, K);
        if (st != MBGLU_OK) return st;
    }
    if (out ? ldo < N : (ldq < N || ldqs < ceil_div(N, kBlk))) return MBGLU_ERR_STRIDE;
    if (!aligned(out, 2) || !aligned(q_scale, 4)) return MBGLU_ERR_ALIGN;
    const int64_t ob = out ? extent(M, N, ldo, 2) : extent(M, N, ldq, 1);
    const int64_t sb = out ? 0 : extent(M, ceil_div(N, kBlk), ldqs, 4);
    const void *o = out ? static_cast<const void *>(out) : q;
    for (const Scaled *in : {&A, &G, &U})
        if (meets(o, ob, *in, K) || meets(q_scale, sb, *in, K)) return MBGLU_ERR_ALIAS;
    if (overlaps(o, ob, q_scale, sb)) return MBGLU_ERR_ALIAS;
    const Fp8Plan plan = fp8_plan(M, N, K, true);
    if (plan.use_tall) {
        mbglu::TallParams p = {};
        p.out = out;
        p.ldo = ldo;
        p.q = q;
        p.ldq = ldq;
        p.qs = q_scale;
        p.ldqs = ldqs;
        mbglu_status st;
        if (q ? tall<2>(plan.tall, A, G, &U, p, M, N, K, stream, &st) : tall<1>(plan.tall, A, G, &U, p, M, N, K, stream, &st))
            return st;
    }
    mbglu::PairMaps maps;
    if (K > 0 && k_major(&maps.a[0], A, K) && k_major(&maps.b[0], G, K) && k_major(&maps.b[1], U, K)) {
        mbglu::Fp8PairParams p = {};
        p.plan = plan.pair;
        p.as = a_scale;
        p.ldas = ldas;
        p.ws[0] = gate_scale;
        p.ldws[0] = ldgs;
        p.ws[1] = up_scale;
        p.ldws[1] = ldus;
        p.wblocks = ceil_div(N, kBlk);
        p.out = out;
        p.ldo = ldo;
        p.out_align = out ? row_align(out, ldo, 2) : 0;
        p.q = q;
        p.ldq = ldq;
        p.q_align = q ? row_align(q, ldq, 1) : 0;
        p.qs = q_scale;
        p.ldqs = ldqs;
        return q ? launch_pair<mbglu::kFp8GluQuant>(p, maps, stream) : launch_pair<mbglu::kFp8Glu>(p, maps, stream);
    }
    mbglu::GenParams p = {};
    p.a[0] = operand(a, lda, a_scale, ldas);
    p.b[0] = operand(gate_w, ld_gate, gate_scale, ldgs);
    p.b[1] = operand(up_w, ld_up, up_scale, ldus);
    p.rows = M;
    p.cols = N;
    p.T = K;
    p.npair = 1;
    p.mode = MBGLU_MODE_FUSED;
    p.out = out;
    p.ldo = ldo;
    p.q = q;
    p.ldq = ldq;
    p.qs = q_scale;
    p.ldqs = ldqs;
    return q ? launch_generic<mbglu::kGenQuant, true>(p, stream) : launch_generic<mbglu::kGenGlu, true>(p, stream);
}

}  // extern "C"

namespace mbglu_host {

void fp8_block_plan(bool dual, int M, int N, int K, int *plan)
{
    const Fp8Plan f = fp8_plan(M, N, K, dual);
    if (f.use_tall) {
        const int tiles = ceil_div(N, mbglu::kTallRows) * ceil_div(M, f.tall.tn), split = f.tall.ks > 1;
        const int got[6] = {1, f.tall.tn, mbglu::kTallRows, split ? 0 : tiles, split ? tiles : 0, f.tall.ks};
        std::copy(got, got + 6, plan);
    } else {
        const int got[6] = {0, mbglu::kPairTile, dual ? 128 : mbglu::kPairTile, f.pair.whole, f.pair.rest, f.pair.splits};
        std::copy(got, got + 6, plan);
    }
}

cudaError_t take_fp8_error(int *w)
{
    cudaError_t e = cudaMemcpyFromSymbol(w, mbglu::g_dense_error, sizeof *w);
    const int zero = 0;
    return e != cudaSuccess ? e : cudaMemcpyToSymbol(mbglu::g_dense_error, &zero, sizeof zero);
}

}  // namespace mbglu_host
