// moe_api.cu -- the mixture-of-experts layer of a decode batch (moe_glu): host-side
// validation, planning and launches.
#include <algorithm>

#include "api_internal.h"
#include "dense_launch.h"
#include "moe_fused.cuh"
#include "moe_generic.cuh"

namespace {

using namespace mbglu_host;

constexpr int kMostBlocks = 160;   // of the fused kernel: what the workspace has room for

// Places of the workspace, in bytes.
struct MoeSpace {
    int64_t counters, logits, ids, weights, gu, y, act, carry, bytes;
};

int64_t act_width(int N) { return (static_cast<int64_t>(N) + 63) / 64 * 64; }

MoeSpace moe_space(int T, int E, int top_k, int N, int K)
{
    MoeSpace s = {};
    const int64_t slots = static_cast<int64_t>(T) * top_k, pad = (T + 15) / 16 * 16;
    s.counters = 0;
    s.logits = MBGLU_MOE_COUNTER_BYTES;
    s.ids = s.logits + padded(static_cast<int64_t>(T) * E * 4);
    s.weights = s.ids + padded(slots * 4);
    s.gu = s.weights + padded(slots * 4);   // the kernels for any alignment: the activation
    s.y = s.gu + padded(slots * 2 * N * 4);
    s.act = s.y + padded(slots * K * 4);
    s.carry = s.act + padded(2 * slots * act_width(N) * 2);
    s.bytes = s.carry + kMostBlocks * pad * 128 * 4;
    return s;
}

bool bad_moe(int T, int E, int top_k, int N, int K)
{
    return T < 0 || T > MBGLU_MAX_M || E < 1 || E > MBGLU_MOE_MAX_EXPERTS || top_k < 1 || top_k > MBGLU_MOE_MAX_TOP_K || top_k > E ||
           bad_sizes(N, K);
}

mbglu_status launch_generic(const mbglu::MoeGeneric &p, cudaStream_t stream)
{
    const auto blocks = [](int64_t n) { return static_cast<unsigned>((n + 7) / 8); };
    const unsigned T = static_cast<unsigned>(p.T), slots = T * static_cast<unsigned>(p.top_k);
    Launch a(dim3(blocks(static_cast<int64_t>(p.T) * p.E)), 256, 0, stream);
    mbglu_status st = launched(cudaLaunchKernelEx(&a.cfg, mbglu::moe_generic_logits, p));
    Launch b(dim3(T), 32, 0, stream);
    if (st == MBGLU_OK) st = launched(cudaLaunchKernelEx(&b.cfg, mbglu::moe_generic_choice, p));
    if (st == MBGLU_OK && p.N > 0) {
        Launch c(dim3(blocks(p.N), slots), 256, 0, stream);
        st = launched(cudaLaunchKernelEx(&c.cfg, mbglu::moe_generic_gated, p));
    }
    if (st == MBGLU_OK && p.K > 0) {
        Launch d(dim3(blocks(p.K), T), 256, 0, stream);
        st = launched(cudaLaunchKernelEx(&d.cfg, mbglu::moe_generic_down, p));
    }
    return st;
}

cudaError_t setup_fused()
{
    return cudaFuncSetAttribute(mbglu::moe_fused_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(mbglu::kMoeSmemMost));
}

bool stackable(const void *p, int64_t stride, int64_t ld, int count)
{
    return copyable(p, ld, 2) && (count == 1 || (stride > 0 && stride % 8 == 0));
}

// The fused kernel; *taken says whether it applies.
mbglu_status launch_fused(const mbglu::MoeGeneric &g, const MoeSpace &space, char *ws, bool *taken, cudaStream_t stream)
{
    *taken = false;
    const int T = g.T, E = g.E, N = g.N, K = g.K;
    if (N == 0 || K == 0 || N % 8 != 0 || K % 8 != 0) return MBGLU_OK;
    if (!copyable(g.h, g.ldh, 2) || !copyable(g.router, g.ldr, 2) || !copyable(g.out, g.ldo, 2) || !stackable(g.gate, g.gate_e, g.ldg, E) ||
        !stackable(g.up, g.up_e, g.ldu, E) || !stackable(g.down, g.down_e, g.ldd, E))
        return MBGLU_OK;
    // units are counted in 32 bits, times the blocks
    const int64_t chosen = std::min<int64_t>(E, static_cast<int64_t>(T) * g.top_k);
    const double units = static_cast<double>(chosen) * std::max(static_cast<double>(ceil_div(N, 64)) * ceil_div(K, 64), 1.0);
    if (units * kMostBlocks > 4.0e9) return MBGLU_OK;
    mbglu::MoeMaps maps;
    mbglu::MoeParams p = {};
    p.pad = (T + 15) / 16 * 16;
    p.act = reinterpret_cast<uint16_t *>(ws + space.act);
    p.act_ld = act_width(N);
    p.act_rows = T * g.top_k;
    if (!encode_stack_map(&maps.gate, g.gate, g.gate_e, g.ldg, E, N, K, 64, 64) || !encode_stack_map(&maps.up, g.up, g.up_e, g.ldu, E, N, K, 64, 64) ||
        !encode_stack_map(&maps.down, g.down, g.down_e, g.ldd, E, K, N, 64, 128) || !encode_tile_map(&maps.h, g.h, g.ldh, T, K, 64, p.pad, 2) ||
        !encode_tile_map(&maps.act, p.act, p.act_ld, 2 * p.act_rows, N, 64, 16, 2))
        return MBGLU_OK;
    static DeviceTable table;
    int sms = 0;
    mbglu_status st = table.get(&sms, setup_fused);
    if (st != MBGLU_OK) return st;
    p.h = g.h;
    p.router = g.router;
    p.ldh = g.ldh;
    p.ldr = g.ldr;
    p.ldo = g.ldo;
    p.out = g.out;
    p.ids = g.user_ids;
    p.weights = g.user_weights;
    p.counters = reinterpret_cast<uint32_t *>(ws + space.counters);
    p.logits = g.logits;
    p.chosen = g.ids;
    p.chosen_weight = g.weights;
    p.gu = reinterpret_cast<float *>(ws + space.gu);
    p.y = reinterpret_cast<float *>(ws + space.y);
    p.carry = reinterpret_cast<float *>(ws + space.carry);
    p.T = T;
    p.E = E;
    p.top_k = g.top_k;
    p.N = N;
    p.K = K;
    p.renormalize = g.renormalize;
    p.stages = mbglu::moe_stages(p.pad);
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeCooperative;   // all blocks resident: they wait for one another
    attr.val.cooperative = 1;
    cfg.gridDim = dim3(static_cast<unsigned>(std::min(sms, kMostBlocks)));
    cfg.blockDim = dim3(mbglu::kMoeThreads);
    cfg.dynamicSmemBytes = mbglu::moe_smem(p.pad);
    cfg.stream = stream;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    *taken = true;
    return launched(cudaLaunchKernelEx(&cfg, mbglu::moe_fused_kernel, p, maps));
}

}  // namespace

extern "C" {

size_t moe_glu_workspace_bytes(int T, int E, int top_k, int N, int K)
{
    if (T == 0 || bad_moe(T, E, top_k, N, K)) return 0;
    return static_cast<size_t>(moe_space(T, E, top_k, N, K).bytes);
}

mbglu_status moe_glu(const mbglu_bf16 *h, int64_t ldh, const mbglu_bf16 *router_w, int64_t ld_router,
                     const mbglu_bf16 *gate_w, int64_t gate_expert, int64_t ld_gate,
                     const mbglu_bf16 *up_w, int64_t up_expert, int64_t ld_up,
                     const mbglu_bf16 *down_w, int64_t down_expert, int64_t ld_down,
                     mbglu_bf16 *out, int64_t ldo, int32_t *ids, float *weights,
                     int T, int E, int top_k, int N, int K, int renormalize,
                     void *workspace, size_t workspace_bytes, cudaStream_t stream)
{
    set_last_variant(0);
    if (bad_moe(T, E, top_k, N, K)) return MBGLU_ERR_SHAPE;
    if (T == 0) return MBGLU_OK;
    if (!workspace || (K > 0 && (!h || !router_w || !out)) || (K > 0 && N > 0 && (!gate_w || !up_w || !down_w))) return MBGLU_ERR_NULL;
    if (K > 0 && (ldh < K || ld_router < K || ldo < K)) return MBGLU_ERR_STRIDE;
    if (K > 0 && N > 0) {
        if (ld_gate < K || ld_up < K || ld_down < N) return MBGLU_ERR_STRIDE;
        if (E > 1 && (gate_expert < 0 || up_expert < 0 || down_expert < 0)) return MBGLU_ERR_STRIDE;
    }
    if (!aligned(h, 2) || !aligned(router_w, 2) || !aligned(gate_w, 2) || !aligned(up_w, 2) || !aligned(down_w, 2) || !aligned(out, 2) ||
        !aligned(ids, 4) || !aligned(weights, 4) || !aligned(workspace, kAlign))
        return MBGLU_ERR_ALIGN;
    const MoeSpace space = moe_space(T, E, top_k, N, K);
    if (workspace_bytes < static_cast<size_t>(space.bytes)) return MBGLU_ERR_SHAPE;
    const int64_t slots = static_cast<int64_t>(T) * top_k;
    const void *ins[5] = {h, router_w, gate_w, up_w, down_w};
    const int64_t inb[5] = {extent(T, K, ldh, 2), extent(E, K, ld_router, 2), K > 0 ? extent3(E, N, K, gate_expert, ld_gate) : 0,
                            K > 0 ? extent3(E, N, K, up_expert, ld_up) : 0, K > 0 ? extent3(E, K, N, down_expert, ld_down) : 0};
    const void *outs[4] = {out, ids, weights, workspace};
    const int64_t outb[4] = {extent(T, K, ldo, 2), ids ? slots * 4 : 0, weights ? slots * 4 : 0, space.bytes};
    for (int i = 0; i < 4; ++i) {
        for (int j = 0; j < 5; ++j)
            if (overlaps(outs[i], outb[i], ins[j], inb[j])) return MBGLU_ERR_ALIAS;
        for (int j = i + 1; j < 4; ++j)
            if (overlaps(outs[i], outb[i], outs[j], outb[j])) return MBGLU_ERR_ALIAS;
    }
    char *ws = static_cast<char *>(workspace);
    mbglu::MoeGeneric p = {};
    p.h = h;
    p.router = router_w;
    p.gate = gate_w;
    p.up = up_w;
    p.down = down_w;
    p.ldh = ldh;
    p.ldr = ld_router;
    p.gate_e = gate_expert;
    p.ldg = ld_gate;
    p.up_e = up_expert;
    p.ldu = ld_up;
    p.down_e = down_expert;
    p.ldd = ld_down;
    p.out = out;
    p.ldo = ldo;
    p.user_ids = ids;
    p.user_weights = weights;
    p.logits = reinterpret_cast<float *>(ws + space.logits);
    p.ids = reinterpret_cast<int32_t *>(ws + space.ids);
    p.weights = reinterpret_cast<float *>(ws + space.weights);
    p.act = reinterpret_cast<float *>(ws + space.gu);
    p.T = T;
    p.E = E;
    p.top_k = top_k;
    p.N = N;
    p.K = K;
    p.renormalize = renormalize;
    bool fused = false;
    mbglu_status st = launch_fused(p, space, ws, &fused, stream);
    if (st == MBGLU_OK && !fused) st = launch_generic(p, stream);
    if (st == MBGLU_OK) set_last_variant(fused ? kMoeFused : kMoeGeneric);
    return st;
}

}  // extern "C"

namespace mbglu_host {

cudaError_t take_moe_error(int *w)
{
    cudaError_t e = cudaMemcpyFromSymbol(w, mbglu::g_dense_error, sizeof *w);
    const int zero = 0;
    return e != cudaSuccess ? e : cudaMemcpyToSymbol(mbglu::g_dense_error, &zero, sizeof zero);
}

}  // namespace mbglu_host
