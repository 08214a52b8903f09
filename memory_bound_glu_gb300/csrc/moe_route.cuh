// moe_route.cuh -- the router of the expert layer: logits whose error is of second order,
// and a warp's choice of the top experts.
//
// An expert is chosen or not, so a logit that is off in its last bit can exchange
// whole experts.  Products of two bf16 numbers are exact in fp32 (down to 2^-134, below which they
// are off by 2^-150 at most); their sum is carried as an unevaluated pair s + c (Knuth's two-sum: s
// the rounded sum, c the sum of the roundings, each of which is exact) and rounded once.  What
// is lost are c's own roundings.  The sums that stand n additions behind the first ones have
// magnitudes of at most S together (S: all products'), their c of n 2^-24 S, and two roundings of
// each lose 2 n 2^-48 S.  With D additions one behind the other, K / 32 of a lane and fewer than 32
// joins of lanes and warps, the pair is off by D (D + 1) 2^-48 S at most.  That is below half a step
// of the logit unless products cancel to less than 2^-10 of S (K = 2048).  It differs with the order
// of the sum, which differs between the kernels and with the number of tokens, so logits that lie
// closer together than that may change places there.  Partial sums beyond fp32's range are
// infinite.  Six additions for each product: 64 rows x 128 experts x 2048 take 118 M operations,
// 3 us of the part's fp32 rate.
#pragma once
#include "glu_math.cuh"
#include "ptx.cuh"

namespace mbglu {

constexpr int kMoeMaxRows = 64, kMoeMaxExperts = 512, kMoeMaxTopK = 16;

// (s, c) += x, exactly but for c's own rounding
__device__ __forceinline__ void two_sum(float &s, float &c, float x)
{
    const float t = __fadd_rn(s, x);
    const float b = __fsub_rn(t, s);
    c = __fadd_rn(c, __fadd_rn(__fsub_rn(s, __fsub_rn(t, b)), __fsub_rn(x, b)));
    s = t;
}

// (s, c) += (s2, c2)
__device__ __forceinline__ void two_sum(float &s, float &c, float s2, float c2)
{
    two_sum(s, c, s2);
    c = __fadd_rn(c, c2);
}

// A pair as one rounded number.  An infinite or NaN sum is the plain one: its roundings are
// infinity - infinity.
__device__ __forceinline__ float pair_value(float s, float c) { return isfinite(s) ? __fadd_rn(s, c) : s; }

// The sum of what a warp's lanes hold, in every lane.
__device__ __forceinline__ void warp_pair_sum(float &s, float &c)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const float s2 = __shfl_xor_sync(0xffffffffu, s, o), c2 = __shfl_xor_sync(0xffffffffu, c, o);
        two_sum(s, c, s2, c2);
    }
}

// Orders floats as integers; -0 counts as 0, NaN (1) is below everything.
__device__ __forceinline__ uint32_t order_key(float x)
{
    if (isnan(x)) return 1;
    const uint32_t u = __float_as_uint(x + 0.0f);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float key_value(uint32_t k)
{
    return k == 1 ? __uint_as_float(0x7fffffffu) : __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k);
}

// One warp: the top_k of `experts` logits, largest first, ties to the lowest index, and
// their softmax weights (over all logits, or over the chosen ones).  Lane j < top_k gets
// the j-th.  A row with a NaN logit gets NaN weights.  PER: logits per lane, 32 PER >=
// experts; logit(e) reads one.
template <int PER, typename F>
__device__ __forceinline__ void warp_top_k(F logit, int experts, int top_k, bool renormalize, int &id, float &weight)
{
    const int lane = threadIdx.x & 31;
    uint32_t key[PER], best = 0, chosen = 0;
    bool nan = false;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        key[i] = i * 32 + lane < experts ? order_key(logit(i * 32 + lane)) : 0u;
        nan = nan || key[i] == 1;
        best = max(best, key[i]);
    }
    nan = __any_sync(0xffffffffu, nan);
    const float top = key_value(__reduce_max_sync(0xffffffffu, best));
    float sum = 0.0f;
    if (!renormalize) {
#pragma unroll
        for (int i = 0; i < PER; ++i)
            if (key[i] != 0) sum += expf(key_value(key[i]) - top);
    }
    id = 0;
    for (int j = 0; j < top_k; ++j) {
        best = 0;
#pragma unroll
        for (int i = 0; i < PER; ++i) best = max(best, key[i]);
        best = __reduce_max_sync(0xffffffffu, best);
        uint32_t at = 0xffffffffu;
#pragma unroll
        for (int i = PER - 1; i >= 0; --i)
            if (key[i] == best) at = static_cast<uint32_t>(i * 32 + lane);
        at = __reduce_min_sync(0xffffffffu, at);
#pragma unroll
        for (int i = 0; i < PER; ++i)
            if (static_cast<uint32_t>(i * 32 + lane) == at) key[i] = 0;
        if (lane == j) {
            id = static_cast<int>(at);
            chosen = best;
        }
    }
    const float e = lane < top_k ? expf(key_value(chosen) - top) : 0.0f;
    if (renormalize) sum = e;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    weight = nan ? __uint_as_float(0x7fffffffu) : e / sum;
}

}  // namespace mbglu
