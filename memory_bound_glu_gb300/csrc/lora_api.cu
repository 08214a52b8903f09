// lora_api.cu -- products with low-rank adapters of many requests beside the shared
// weights (glu_lora, linear_lora): host-side validation, planning and launches.
#include <algorithm>

#include "api_internal.h"
#include "dense_launch.h"
#include "lora_generic.cuh"

namespace {

using namespace mbglu_host;

constexpr int64_t kAlign = 256;
int64_t padded(int64_t bytes) { return (bytes + kAlign - 1) / kAlign * kAlign; }

int64_t lora_space(int sides, int M, int R) { return padded(static_cast<int64_t>(M) * sides * R * 4); }

bool bad_rank(int adapters, int R) { return adapters < 0 || adapters > kMostSize || R < 0 || R > MBGLU_LORA_MAX_RANK; }

// bytes from the first element of [count][rows][cols] to the end of its last
int64_t extent3(int64_t count, int64_t rows, int64_t cols, int64_t stride, int64_t ld)
{
    return count <= 0 || rows <= 0 || cols <= 0 ? 0 : (count - 1) * stride * 2 + extent(rows, cols, ld, 2);
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
    const int64_t need = adapted ? lora_space(SIDES, M, R) : 0;
    if (workspace_bytes < static_cast<size_t>(need)) return MBGLU_ERR_SHAPE;
    const void *outs[2] = {p.out, workspace};
    const int64_t outb[2] = {extent(M, N, p.ldo, 2), need};
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
    p.p = static_cast<float *>(workspace);
    mbglu_status st = MBGLU_OK;
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
    return static_cast<size_t>(lora_space(2, M, R));
}

size_t linear_lora_workspace_bytes(int M, int N, int K, int adapters, int R)
{
    if (bad_sizes(M, N, K) || N > INT32_MAX / 2 || bad_rank(adapters, R) || std::min({M, N, K, adapters, R}) == 0) return 0;
    return static_cast<size_t>(lora_space(1, M, R));
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
