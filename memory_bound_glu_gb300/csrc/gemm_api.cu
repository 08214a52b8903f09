// gemm_api.cu -- the gated block at any number of rows in bf16 (glu_gemm) and
// its backward pass (glu_gemm_backward): host-side validation, planning and
// launches.
#include <algorithm>
#include <mutex>

#include "api_internal.h"
#include "dense_generic.cuh"
#include "dense_launch.h"

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

}  // namespace

extern "C" {

mbglu_status glu_gemm(const mbglu_bf16 *h, int64_t ldh, const mbglu_bf16 *gate_w, int64_t ld_gate,
                      const mbglu_bf16 *up_w, int64_t ld_up, mbglu_bf16 *out, int64_t ldo, float *gu, int64_t ldgu,
                      int M, int N, int K, mbglu_mode mode, cudaStream_t stream)
{
    set_last_variant(0);
    if (mode != MBGLU_MODE_FUSED && mode != MBGLU_MODE_HF) return MBGLU_ERR_MODE;
    if (M < 0 || N < 0 || K < 0 || N > INT32_MAX / 2) return MBGLU_ERR_SHAPE;
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
    // few rows: the decode kernels, which hand out no g and u
    if (M <= MBGLU_MAX_M && !gu)
        return glu_gemv(h, ldh, gate_w, ld_gate, up_w, ld_up, out, ldo, M, N, K, mode, stream);
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
    if (M <= 0 || N <= 0 || K <= 0) return 0;
    return static_cast<size_t>(grad_bytes(M, N));
}

mbglu_status glu_gemm_backward(const mbglu_bf16 *h, int64_t ldh, const mbglu_bf16 *gate_w, int64_t ld_gate,
                               const mbglu_bf16 *up_w, int64_t ld_up, const mbglu_bf16 *dout, int64_t ldd,
                               const float *gu, int64_t ldgu, mbglu_bf16 *grad_h, int64_t ldgh, mbglu_bf16 *grad_gate,
                               int64_t ldgg, mbglu_bf16 *grad_up, int64_t ldgu_w, int M, int N, int K,
                               void *workspace, size_t workspace_bytes, cudaStream_t stream)
{
    set_last_variant(0);
    set_last_backward_path(0);
    if (M < 0 || N < 0 || K < 0 || N > INT32_MAX / 2) return MBGLU_ERR_SHAPE;
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
    mbglu_status st = launch_generic<mbglu::kGenGrad, true>(p, stream);
    if (st == MBGLU_OK && want_h) {   // dG Wg + dU Wu
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
    if (st == MBGLU_OK) {
        set_last_variant(kGemmBackward);
        set_last_backward_path(5);
    }
    return st;
}

}  // extern "C"

namespace mbglu_host {

__device__ int g_gemm_error;

cudaError_t take_gemm_error(int *w)
{
    cudaError_t e = cudaMemcpyFromSymbol(w, g_gemm_error, sizeof *w);
    const int zero = 0;
    return e != cudaSuccess ? e : cudaMemcpyToSymbol(g_gemm_error, &zero, sizeof zero);
}

}  // namespace mbglu_host
