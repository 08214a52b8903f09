// gemm_api.cu -- the gated block at any number of rows in bf16 (glu_gemm) and
// its backward pass (glu_gemm_backward): host-side validation, planning and
// launches.
#include <algorithm>

#include "api_internal.h"
#include "dense_generic.cuh"
#include "dense_launch.h"
#include "glu_grad.cuh"
#include "pair_gemm.cuh"
#include "pair_plan.h"
#include "pair_tall.cuh"

namespace {

using namespace mbglu_host;

mbglu::GenOperand operand(const void *p, int64_t s_out, int64_t s_t)
{
    mbglu::GenOperand o = {};
    o.p = p;
    o.s_out = s_out;
    o.s_t = s_t;
    return o;
}

template <int EPI, bool DUAL>
mbglu_status launch_generic(const mbglu::GenParams &p, cudaStream_t stream)
{
    Launch l(mbglu::gen_grid(p.rows, p.cols), 256, 0, stream);
    return launched(cudaLaunchKernelEx(&l.cfg, mbglu::dense_generic_kernel<EPI, false, DUAL>, p));
}

// ---- the CTA-pair kernels --------------------------------------------------------

template <int EPI, int MODE, bool A_MN, bool B_MN>
cudaError_t allow_pair()
{
    return cudaFuncSetAttribute(mbglu::pair_gemm_kernel<EPI, MODE, A_MN, B_MN>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                static_cast<int>(mbglu::kPairSmem));
}

cudaError_t setup_pair()
{
    cudaError_t e = allow_pair<mbglu::kPairGlu, mbglu::kPairDual, false, false>();
    if (e == cudaSuccess) e = allow_pair<mbglu::kPairGrad, mbglu::kPairDual, false, false>();
    if (e == cudaSuccess) e = allow_pair<mbglu::kPairPlain, mbglu::kPairSum, false, true>();
    if (e == cudaSuccess) e = allow_pair<mbglu::kPairPlain, mbglu::kPairStack, true, true>();
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(mbglu::pair_tall_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(mbglu::kPairSmem));
    return e;
}

mbglu_status sm_count(int *n)
{
    static DeviceTable table;
    return table.get(n, setup_pair);
}

bool k_major(mbglu::TensorMap *m, const void *p, int64_t ld, int rows, int T, int box_rows = 128)
{
    return encode_tile_map(m, p, ld, rows, T, 64, box_rows, 2);
}

// [T][cols], cols the output's index
bool mn_major(mbglu::TensorMap *m, const void *p, int64_t ld, int T, int cols)
{
    return encode_tile_map(m, p, ld, T, cols, 64, 64, 2);
}

template <int EPI, int MODE, bool A_MN, bool B_MN>
mbglu_status launch_pair(const mbglu::PairParams &p, const mbglu::PairMaps &maps, cudaStream_t stream)
{
    int sms = 0;
    const mbglu_status st = sm_count(&sms);
    if (st != MBGLU_OK) return st;
    Launch l(dim3(static_cast<unsigned>(2 * std::min(std::max(sms / 2, 1), p.plan.ntiles))), mbglu::kPairThreads, mbglu::kPairSmem,
             stream, 2);
    return launched(cudaLaunchKernelEx(&l.cfg, mbglu::pair_gemm_kernel<EPI, MODE, A_MN, B_MN>, p, maps));
}

constexpr int kDecodeRows = 16;   // glu_gemv's, at any alignment

// Tokens per tile of pair_tall_kernel, or 0 where pair_gemm_kernel is estimated to
// be faster.  From the sizes alone.  The constants (ns) are fitted to 600 measured
// calls in chains: seven shapes, 65 to 1000 rows, every tn.  There the choice is
// within 1% of the fastest on average, 7% at worst, never slower than
// pair_gemm_kernel and 24% faster on average (K = 2560, N = 9728 at M = 333: 27.9 us
// against 31.2; K = 1000, N = 2504: 9.2 and 11.3; K = 4096, N = 300: 13.0 and 22.9).
// Outside the fit, over N = 300 to 14336 and K = 264 to 9728: at 17 to 64 rows (175
// calls) within 4% of the fastest of tn = 32 to 128, and pair_gemm_kernel takes 1.05 to
// 2.2 times as long; at 1024 to 8192 rows (245 calls) never slower than
// pair_gemm_kernel and 25% faster on average where it takes a tn.  Where it keeps
// pair_gemm_kernel there, a tn would be faster in a third of the calls, by 7% on average
// (3000 x 2560 -> 2560: 50.5 us, 44.5 with tn = 160; 3000 x 264 -> 300: 8.4 and 6.5 with 128).
// The estimate ranks kernels and is no time: it knows nothing of the weights' bytes,
// and tall_outputs' narrower tiles are chosen after it.
int tall_tokens(int M, int N, int K)
{
    const int64_t chunks = ceil_div(K, 64), nt = ceil_div(N, 128), tiles = nt * ceil_div(M, mbglu::kPairTile);
    int64_t best = 5760 + (tiles + kPairs - 1) / kPairs * chunks * (253 + 88 * std::min<int64_t>(tiles, kPairs) / kPairs);
    int tn = 0;
    for (int t = 32; t < mbglu::kPairTile; t += 32) {
        const int64_t n = nt * ceil_div(M, t);
        const int64_t round = chunks * (77 + 59 * std::min<int64_t>(n, kPairs) / kPairs) + chunks * t * 7 / 10 + t * 31 / 2;
        const int64_t ns = 4240 + (n + kPairs - 1) / kPairs * round;
        if (ns < best) {
            best = ns;
            tn = t;
        }
    }
    return tn;
}

// Outputs per tile: 80 or 96 where that needs no more rounds over the SM pairs than
// 128 does, so that a round brings fewer weights.  K = 4096, N = 11008: 34.6 us with 80
// against 40.0 with 128 at M = 17, 37.7 and 42.6 at 100, 39.0 and 43.4 at 160; where the
// least such width is 112, up to 2.6% slower, so not there; nor narrower than 80 (K =
// 1024, N = 640 at M = 160: 4.9 us, 5.2 with 64).
int tall_outputs(int M, int N, int tn)
{
    const int64_t tt = ceil_div(M, tn), places = (ceil_div(N, 128) * tt + kPairs - 1) / kPairs * kPairs;
    for (const int wt : {80, 96})
        if (ceil_div(N, wt) * tt <= places) return wt;
    return 128;
}

mbglu_status launch_pair_tall(const mbglu::PairTallParams &p, const mbglu::PairMaps &maps, cudaStream_t stream)
{
    int sms = 0;
    const mbglu_status st = sm_count(&sms);
    if (st != MBGLU_OK) return st;
    Launch l(dim3(static_cast<unsigned>(2 * std::min(std::max(sms / 2, 1), p.ntiles))), mbglu::kPairThreads, mbglu::kPairSmem, stream, 2);
    return launched(cudaLaunchKernelEx(&l.cfg, mbglu::pair_tall_kernel, p, maps));
}

// grad_h [M, K] over 2 N; grad_gate and grad_up [N, K] over M
mbglu::PairPlan grad_h_plan(int M, int N, int K)
{
    const int chunks = ceil_div(N, 64);
    return pair_plan(M, K, 256, 1, chunks, 2 * chunks, true);
}
mbglu::PairPlan grad_w_plan(int M, int N, int K) { return pair_plan(N, K, 256, 2, 0, ceil_div(M, 64), true); }

}  // namespace

extern "C" {

mbglu_status glu_gemm(const mbglu_bf16 *h, int64_t ldh, const mbglu_bf16 *gate_w, int64_t ld_gate,
                      const mbglu_bf16 *up_w, int64_t ld_up, mbglu_bf16 *out, int64_t ldo, float *gu, int64_t ldgu,
                      int M, int N, int K, mbglu_mode mode, cudaStream_t stream)
{
    set_last_variant(0);
    if (mode != MBGLU_MODE_FUSED && mode != MBGLU_MODE_HF) return MBGLU_ERR_MODE;
    if (bad_sizes(M, N, K) || N > INT32_MAX / 2) return MBGLU_ERR_SHAPE;
    if (M == 0 || N == 0) return MBGLU_OK;
    if (!out || (K > 0 && (!h || !gate_w || !up_w))) return MBGLU_ERR_NULL;
    if (ldo < N || (gu && ldgu < 2 * static_cast<int64_t>(N)) || (K > 0 && (ldh < K || ld_gate < K || ld_up < K)))
        return MBGLU_ERR_STRIDE;
    if (!aligned(out, 2) || !aligned(gu, 4) || !aligned(h, 2) || !aligned(gate_w, 2) || !aligned(up_w, 2))
        return MBGLU_ERR_ALIGN;
    const int64_t ob = extent(M, N, ldo, 2), gb = gu ? extent(M, 2 * static_cast<int64_t>(N), ldgu, 4) : 0;
    if (overlaps(out, ob, gu, gb)) return MBGLU_ERR_ALIAS;
    if (K > 0) {
        const void *ins[3] = {h, gate_w, up_w};
        const int64_t inb[3] = {extent(M, K, ldh, 2), extent(N, K, ld_gate, 2), extent(N, K, ld_up, 2)};
        for (int i = 0; i < 3; ++i)
            if (overlaps(out, ob, ins[i], inb[i]) || overlaps(gu, gb, ins[i], inb[i])) return MBGLU_ERR_ALIAS;
    }
    // few rows: the decode kernels, which hand out no g and u.  From 17 rows on
    // pair_tall_kernel is faster wherever it applies: 19.1 us against 23.3 at 17 rows
    // and 19.7 against 29.4 at 64 (K = 2560, N = 9728), 6.5 against 20.9 at 64 (K = 1000,
    // N = 2504); at 16, 18.8 and 20.1, 10.1 and 6.5 (K = 2560, N = 1000).
    const bool fast = K > 0 && copyable(h, ldh, 2) && copyable(gate_w, ld_gate, 2) && copyable(up_w, ld_up, 2);
    if (!gu && (M <= kDecodeRows || (M <= MBGLU_MAX_M && !fast)))
        return glu_gemv(h, ldh, gate_w, ld_gate, up_w, ld_up, out, ldo, M, N, K, mode, stream);
    mbglu::PairMaps maps;
    const int tn = fast ? tall_tokens(M, N, K) : 0;
    const int wt = tn ? tall_outputs(M, N, tn) : 0;
    if (tn && k_major(&maps.a[0], gate_w, ld_gate, N, K, wt / 2) && k_major(&maps.a[1], up_w, ld_up, N, K, wt / 2) &&
        k_major(&maps.b[0], h, ldh, M, K, tn / 2)) {
        mbglu::PairTallParams q = {};
        q.M = M;
        q.N = N;
        q.nchunk = ceil_div(K, 64);
        q.tn = tn;
        q.ttiles = ceil_div(M, tn);
        q.ntiles = q.ttiles * ceil_div(N, wt);
        q.wt = wt;
        q.mode = static_cast<int>(mode);
        q.out = out;
        q.ldo = ldo;
        q.gu = gu;
        q.ldgu = ldgu;
        const mbglu_status st = launch_pair_tall(q, maps, stream);
        if (st == MBGLU_OK) set_last_variant(kPairGemm);
        return st;
    }
    if (fast && k_major(&maps.a[0], h, ldh, M, K) &&
        k_major(&maps.b[0], gate_w, ld_gate, N, K) && k_major(&maps.b[1], up_w, ld_up, N, K)) {
        mbglu::PairParams q = {};
        q.plan = pair_plan(M, N, 128, 1, 0, ceil_div(K, 64), false);
        q.mode = static_cast<int>(mode);
        q.out[0] = out;
        q.ldo[0] = ldo;
        q.out_align[0] = row_align(out, ldo, 2);
        q.gu = gu;
        q.ldgu = ldgu;
        q.gu_align = gu ? row_align(gu, ldgu, 4) : 0;
        q.gu_align_u = gu ? row_align(gu + N, ldgu, 4) : 0;
        const mbglu_status st = launch_pair<mbglu::kPairGlu, mbglu::kPairDual, false, false>(q, maps, stream);
        if (st == MBGLU_OK) set_last_variant(kPairGemm);
        return st;
    }
    mbglu::GenParams p = {};
    p.a[0] = operand(h, ldh, 1);
    p.b[0] = operand(gate_w, ld_gate, 1);
    p.b[1] = operand(up_w, ld_up, 1);
    p.rows = M;
    p.cols = N;
    p.T = K;
    p.npair = 1;
    p.mode = static_cast<int>(mode);
    p.out = out;
    p.ldo = ldo;
    p.gu = gu;
    p.ldgu = ldgu;
    const mbglu_status st = launch_generic<mbglu::kGenGlu, true>(p, stream);
    if (st == MBGLU_OK) set_last_variant(kGemmGeneric);
    return st;
}

// dG and dU in bf16, [M][width] each, width = N rounded up so that every row
// starts on 128 bytes
static int64_t grad_width(int N) { return (static_cast<int64_t>(N) + 63) / 64 * 64; }
static int64_t grad_bytes(int M, int N) { return (2 * static_cast<int64_t>(M) * grad_width(N) * 2 + 255) / 256 * 256; }

size_t glu_gemm_backward_workspace_bytes(int M, int N, int K)
{
    if (M <= 0 || N <= 0 || K <= 0 || bad_sizes(M, N, K)) return 0;
    // the two products' partial sums, one after the other
    return static_cast<size_t>(grad_bytes(M, N) + std::max(part_bytes(grad_h_plan(M, N, K)), part_bytes(grad_w_plan(M, N, K))));
}

mbglu_status glu_gemm_backward(const mbglu_bf16 *h, int64_t ldh, const mbglu_bf16 *gate_w, int64_t ld_gate,
                               const mbglu_bf16 *up_w, int64_t ld_up, const mbglu_bf16 *dout, int64_t ldd,
                               const float *gu, int64_t ldgu, mbglu_bf16 *grad_h, int64_t ldgh, mbglu_bf16 *grad_gate,
                               int64_t ldgg, mbglu_bf16 *grad_up, int64_t ldgu_w, int M, int N, int K,
                               void *workspace, size_t workspace_bytes, cudaStream_t stream)
{
    set_last_variant(0);
    set_last_backward_path(0);
    if (bad_sizes(M, N, K) || N > INT32_MAX / 2) return MBGLU_ERR_SHAPE;
    const bool want_h = grad_h != nullptr, want_w = grad_gate != nullptr || grad_up != nullptr;
    if (want_w && (!grad_gate || !grad_up)) return MBGLU_ERR_NULL;
    if (K == 0) return MBGLU_OK;   // every gradient has K columns
    const bool full = M > 0 && N > 0;
    if (full && (!h || !gate_w || !up_w || !dout || !workspace)) return MBGLU_ERR_NULL;
    if ((M > 0 && want_h && ldgh < K) || (N > 0 && want_w && (ldgg < K || ldgu_w < K))) return MBGLU_ERR_STRIDE;
    if (full && (ldh < K || ld_gate < K || ld_up < K || ldd < N || (gu && ldgu < 2 * static_cast<int64_t>(N))))
        return MBGLU_ERR_STRIDE;
    if (!aligned(h, 2) || !aligned(gate_w, 2) || !aligned(up_w, 2) || !aligned(dout, 2) || !aligned(grad_h, 2) ||
        !aligned(grad_gate, 2) || !aligned(grad_up, 2) || !aligned(workspace, 256) || !aligned(gu, 4))
        return MBGLU_ERR_ALIGN;
    const size_t need = glu_gemm_backward_workspace_bytes(M, N, K);
    if (full && workspace_bytes < need) return MBGLU_ERR_SHAPE;
    const void *ins[5] = {h, gate_w, up_w, dout, gu};
    const int64_t inb[5] = {full ? extent(M, K, ldh, 2) : 0, full ? extent(N, K, ld_gate, 2) : 0,
                            full ? extent(N, K, ld_up, 2) : 0, full ? extent(M, N, ldd, 2) : 0,
                            full && gu ? extent(M, 2 * static_cast<int64_t>(N), ldgu, 4) : 0};
    const void *outs[4] = {grad_h, grad_gate, grad_up, workspace};
    const int64_t outb[4] = {want_h ? extent(M, K, ldgh, 2) : 0, want_w ? extent(N, K, ldgg, 2) : 0,
                             want_w ? extent(N, K, ldgu_w, 2) : 0, full ? static_cast<int64_t>(need) : 0};
    for (int i = 0; i < 4; ++i) {
        for (int j = 0; j < 5; ++j)
            if (overlaps(outs[i], outb[i], ins[j], inb[j])) return MBGLU_ERR_ALIAS;
        for (int j = i + 1; j < 4; ++j)
            if (overlaps(outs[i], outb[i], outs[j], outb[j])) return MBGLU_ERR_ALIAS;
    }
    if ((M == 0 && N == 0) || (!want_h && !want_w)) return MBGLU_OK;
    if (!full) {   // N == 0: grad_h = 0; M == 0: grad_gate = grad_up = 0
        cudaError_t e = cudaSuccess;
        if (N == 0 && want_h)
            e = cudaMemset2DAsync(grad_h, static_cast<size_t>(ldgh) * 2, 0, static_cast<size_t>(K) * 2, M, stream);
        if (M == 0 && want_w) {
            e = cudaMemset2DAsync(grad_gate, static_cast<size_t>(ldgg) * 2, 0, static_cast<size_t>(K) * 2, N, stream);
            if (e == cudaSuccess)
                e = cudaMemset2DAsync(grad_up, static_cast<size_t>(ldgu_w) * 2, 0, static_cast<size_t>(K) * 2, N, stream);
        }
        return launched(e);
    }
    const int64_t W = grad_width(N);
    uint16_t *dG = static_cast<uint16_t *>(workspace), *dU = dG + static_cast<int64_t>(M) * W;

    float *part = reinterpret_cast<float *>(static_cast<char *>(workspace) + grad_bytes(M, N));
    const bool fast_h = copyable(h, ldh, 2), fast_w = copyable(gate_w, ld_gate, 2) && copyable(up_w, ld_up, 2);
    mbglu_status st = MBGLU_OK;
    mbglu::PairMaps maps;
    int path = 4;

    // 1) dG, dU: from g and u as the forward kept them, or both products again
    if (gu) {
        const int vec = N % 8 == 0 && aligned(gu, 16) && ldgu % 4 == 0 && aligned(dout, 16) && ldd % 8 == 0;
        const int64_t work = static_cast<int64_t>(M) * (vec ? N / 8 : N);
        Launch l(dim3(static_cast<unsigned>(std::min<int64_t>((work + 255) / 256, 1 << 20))), 256, 0, stream);
        st = launched(cudaLaunchKernelEx(&l.cfg, mbglu::glu_grad_kernel, gu, ldgu, static_cast<const uint16_t *>(dout), ldd, dG, dU,
                                         W, M, N, vec));
    } else if (fast_h && fast_w && k_major(&maps.a[0], h, ldh, M, K) && k_major(&maps.b[0], gate_w, ld_gate, N, K) &&
               k_major(&maps.b[1], up_w, ld_up, N, K)) {
        mbglu::PairParams q = {};
        q.plan = pair_plan(M, N, 128, 1, 0, ceil_div(K, 64), false);
        q.out[0] = dG;
        q.out[1] = dU;
        q.ldo[0] = q.ldo[1] = W;
        q.out_align[0] = row_align(dG, W, 2);
        q.out_align[1] = row_align(dU, W, 2);
        q.dout = dout;
        q.ldd = ldd;
        q.dout_align = row_align(dout, ldd, 2);
        st = launch_pair<mbglu::kPairGrad, mbglu::kPairDual, false, false>(q, maps, stream);
    } else {
        path = 5;
        mbglu::GenParams p = {};
        p.a[0] = operand(h, ldh, 1);
        p.b[0] = operand(gate_w, ld_gate, 1);
        p.b[1] = operand(up_w, ld_up, 1);
        p.rows = M;
        p.cols = N;
        p.T = K;
        p.npair = 1;
        p.dout = dout;
        p.ldd = ldd;
        p.out = dG;
        p.out2 = dU;
        p.ldo = W;
        st = launch_generic<mbglu::kGenGrad, true>(p, stream);
    }

    // 2) grad_h = dG Wg + dU Wu: one sum over 2N
    if (st == MBGLU_OK && want_h && fast_w && k_major(&maps.a[0], dG, W, M, N) && k_major(&maps.a[1], dU, W, M, N) &&
        mn_major(&maps.b[0], gate_w, ld_gate, N, K) && mn_major(&maps.b[1], up_w, ld_up, N, K)) {
        mbglu::PairParams q = {};
        q.plan = grad_h_plan(M, N, K);
        q.out[0] = grad_h;
        q.ldo[0] = ldgh;
        q.out_align[0] = row_align(grad_h, ldgh, 2);
        q.part = part;
        st = launch_pair<mbglu::kPairPlain, mbglu::kPairSum, false, true>(q, maps, stream);
        if (st == MBGLU_OK) st = launch_join(q.plan, part, q.out, q.ldo, stream);
    } else if (st == MBGLU_OK && want_h) {
        path = 5;
        mbglu::GenParams q = {};
        q.a[0] = operand(dG, W, 1);
        q.a[1] = operand(dU, W, 1);
        q.b[0] = operand(gate_w, 1, ld_gate);
        q.b[1] = operand(up_w, 1, ld_up);
        q.rows = M;
        q.cols = K;
        q.T = N;
        q.npair = 2;
        q.out = grad_h;
        q.ldo = ldgh;
        st = launch_generic<mbglu::kGenPlain, false>(q, stream);
    }

    // 3) grad_gate = dG^T h, grad_up = dU^T h: the tiles of both in one launch
    if (st == MBGLU_OK && want_w && fast_h && mn_major(&maps.a[0], dG, W, M, N) && mn_major(&maps.a[1], dU, W, M, N) &&
        mn_major(&maps.b[0], h, ldh, M, K)) {
        mbglu::PairParams q = {};
        q.plan = grad_w_plan(M, N, K);
        q.part = part;
        q.out[0] = grad_gate;
        q.out[1] = grad_up;
        q.ldo[0] = ldgg;
        q.ldo[1] = ldgu_w;
        q.out_align[0] = row_align(grad_gate, ldgg, 2);
        q.out_align[1] = row_align(grad_up, ldgu_w, 2);
        st = launch_pair<mbglu::kPairPlain, mbglu::kPairStack, true, true>(q, maps, stream);
        if (st == MBGLU_OK) st = launch_join(q.plan, part, q.out, q.ldo, stream);
    } else if (want_w) {
        path = 5;
        for (int i = 0; st == MBGLU_OK && want_w && i < 2; ++i) {   // dG^T h, dU^T h
            mbglu::GenParams q = {};
            q.a[0] = operand(i ? dU : dG, 1, W);
            q.b[0] = operand(h, 1, ldh);
            q.rows = N;
            q.cols = K;
            q.T = M;
            q.npair = 1;
            q.out = i ? grad_up : grad_gate;
            q.ldo = i ? ldgu_w : ldgg;
            st = launch_generic<mbglu::kGenPlain, false>(q, stream);
        }
    }
    if (st == MBGLU_OK) {
        set_last_variant(kGemmBackward);
        set_last_backward_path(path);
    }
    return st;
}

mbglu_status mbglu_block_plan(int product, int M, int N, int K, int *plan)
{
    if (!plan) return MBGLU_ERR_NULL;
    if (product < MBGLU_PRODUCT_GLU_GEMM || product > MBGLU_PRODUCT_MATMUL_FP8) return MBGLU_ERR_MODE;
    if (bad_sizes(M, N, K) || std::min({M, N, K}) < 1 || N > INT32_MAX / 2) return MBGLU_ERR_SHAPE;
    // tiles are counted in 32 bits, ranges included (the smallest: 16 x 64 in 16 ranges)
    const int64_t rows = product == MBGLU_PRODUCT_GRAD_W ? N : M;
    const int64_t cols = product == MBGLU_PRODUCT_GRAD_H || product == MBGLU_PRODUCT_GRAD_W ? K : N;
    if (rows / 16 + 1 > INT32_MAX / (16 * (cols / 64 + 1))) return MBGLU_ERR_SHAPE;
    if (product >= MBGLU_PRODUCT_GLU_FP8) {
        fp8_block_plan(product == MBGLU_PRODUCT_GLU_FP8, M, N, K, plan);
        return MBGLU_OK;
    }
    const int tn = product == MBGLU_PRODUCT_GLU_GEMM ? tall_tokens(M, N, K) : 0;
    if (tn) {
        const int wt = tall_outputs(M, N, tn);
        const int got[6] = {1, tn, wt, ceil_div(N, wt) * ceil_div(M, tn), 0, 1};
        std::copy(got, got + 6, plan);
        return MBGLU_OK;
    }
    const mbglu::PairPlan p = product == MBGLU_PRODUCT_GRAD_H   ? grad_h_plan(M, N, K)
                              : product == MBGLU_PRODUCT_GRAD_W ? grad_w_plan(M, N, K)
                                                                : pair_plan(M, N, 128, 1, 0, ceil_div(K, 64), false);
    const int got[6] = {0, mbglu::kPairTile, product == MBGLU_PRODUCT_GLU_GEMM ? 128 : mbglu::kPairTile, p.whole, p.rest, p.splits};
    std::copy(got, got + 6, plan);
    return MBGLU_OK;
}

}  // extern "C"

namespace mbglu_host {

// This unit's word, or else one of the units whose rows choose weights of their own.
cudaError_t take_gemm_error(int *w)
{
    cudaError_t e = cudaMemcpyFromSymbol(w, mbglu::g_dense_error, sizeof *w);
    const int zero = 0;
    if (e == cudaSuccess) e = cudaMemcpyToSymbol(mbglu::g_dense_error, &zero, sizeof zero);
    for (cudaError_t (*take)(int *) : {take_lora_error, take_moe_error}) {
        int x = 0;
        if (e == cudaSuccess) e = take(&x);
        if (*w == 0) *w = x;
    }
    return e;
}

}  // namespace mbglu_host
