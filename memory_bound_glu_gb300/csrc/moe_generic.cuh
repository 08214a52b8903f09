// moe_generic.cuh -- the expert layer for operands that tensor copies cannot take
// (odd strides, sizes or base addresses) and for empty sums: the kernels that are right
// for every case.  A warp per logit, per token's choice, per gated product of a chosen
// expert and per output; fp32 sums, the activation kept in fp32, one rounding at the end.
#pragma once
#include "moe_route.cuh"

namespace mbglu {

struct MoeGeneric {
    const uint16_t *h, *router, *gate, *up, *down;
    int64_t ldh, ldr, gate_e, ldg, up_e, ldu, down_e, ldd, ldo;
    uint16_t *out;
    int32_t *ids, *user_ids;   // workspace [T][top_k]; the caller's, or null
    float *weights, *user_weights, *logits, *act;
    int T, E, top_k, N, K, renormalize;
};

static __global__ void __launch_bounds__(256) moe_generic_logits(const MoeGeneric p)
{
    grid_dependency_wait();
    grid_launch_dependents();
    const int64_t i = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
    if (i >= static_cast<int64_t>(p.T) * p.E) return;
    const int t = static_cast<int>(i / p.E), e = static_cast<int>(i % p.E);
    const uint16_t *a = p.h + t * p.ldh, *b = p.router + e * p.ldr;
    float s = 0.0f, c = 0.0f;
    for (int k = threadIdx.x & 31; k < p.K; k += 32) two_sum(s, c, __fmul_rn(bf16_to_f32(a[k]), bf16_to_f32(b[k])));
    warp_pair_sum(s, c);
    if ((threadIdx.x & 31) == 0) p.logits[i] = pair_value(s, c);
}

static __global__ void __launch_bounds__(32) moe_generic_choice(const MoeGeneric p)
{
    grid_dependency_wait();
    grid_launch_dependents();
    const int t = blockIdx.x, lane = threadIdx.x;
    int id;
    float w;
    warp_top_k<kMoeMaxExperts / 32>([&](int e) { return p.logits[t * p.E + e]; }, p.E, p.top_k, p.renormalize != 0, id, w);
    if (lane < p.top_k) {
        p.ids[t * p.top_k + lane] = id;
        p.weights[t * p.top_k + lane] = w;
        if (p.user_ids) p.user_ids[t * p.top_k + lane] = id;
        if (p.user_weights) p.user_weights[t * p.top_k + lane] = w;
    }
}

// act[slot][n] = SiLU(h gate_w[e][n]) (h up_w[e][n]); slot = t top_k + j
static __global__ void __launch_bounds__(256) moe_generic_gated(const MoeGeneric p)
{
    grid_dependency_wait();
    grid_launch_dependents();
    const int slot = blockIdx.y, lane = threadIdx.x & 31;
    const int64_t n = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
    if (n >= p.N) return;
    const int e = p.ids[slot];
    const uint16_t *x = p.h + slot / p.top_k * p.ldh, *a = p.gate + e * p.gate_e + n * p.ldg, *b = p.up + e * p.up_e + n * p.ldu;
    float g = 0.0f, u = 0.0f;
    for (int k = lane; k < p.K; k += 32) {
        const float v = bf16_to_f32(x[k]);
        g = fmaf(v, bf16_to_f32(a[k]), g);
        u = fmaf(v, bf16_to_f32(b[k]), u);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        g += __shfl_xor_sync(0xffffffffu, g, o);
        u += __shfl_xor_sync(0xffffffffu, u, o);
    }
    if (lane == 0) p.act[static_cast<int64_t>(slot) * p.N + n] = silu_f32(g) * u;
}

static __global__ void __launch_bounds__(256) moe_generic_down(const MoeGeneric p)
{
    grid_dependency_wait();
    grid_launch_dependents();
    const int t = blockIdx.y, lane = threadIdx.x & 31;
    const int64_t k = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
    if (k >= p.K) return;
    float out = 0.0f;
    for (int j = 0; j < p.top_k; ++j) {
        const int slot = t * p.top_k + j;
        const uint16_t *d = p.down + p.ids[slot] * p.down_e + k * p.ldd;
        const float *a = p.act + static_cast<int64_t>(slot) * p.N;
        float y = 0.0f;
        for (int n = lane; n < p.N; n += 32) y = fmaf(a[n], bf16_to_f32(d[n]), y);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) y += __shfl_xor_sync(0xffffffffu, y, o);
        out = fmaf(p.weights[slot], y, out);
    }
    if (lane == 0) p.out[t * p.ldo + k] = f32_to_bf16(out);
}

}  // namespace mbglu
