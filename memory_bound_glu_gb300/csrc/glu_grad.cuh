// glu_grad.cuh -- the backward's element-wise step where the forward kept g and u.
#pragma once

#include "dense_common.cuh"

namespace mbglu {

// dG, dU (bf16, [rows][ldo]) from g and u as the forward kept them: one pass,
// 8 columns per thread where everything lies on 16 bytes (vec).
__global__ void __launch_bounds__(256) glu_grad_kernel(const float *gu, int64_t ldgu, const uint16_t *dout, int64_t ldd,
                                                       uint16_t *dg, uint16_t *du, int64_t ldo, int rows, int cols, int vec)
{
    grid_dependency_wait();
    grid_launch_dependents();
    const int per = vec ? cols / 8 : cols;
    const int64_t total = static_cast<int64_t>(rows) * per;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < total; i += static_cast<int64_t>(gridDim.x) * 256) {
        const int64_t m = i / per;
        const int c = static_cast<int>(i - m * per);
        if (vec) {
            const float4 *pg = reinterpret_cast<const float4 *>(gu + m * ldgu) + 2 * c;
            const float4 *pu = reinterpret_cast<const float4 *>(gu + m * ldgu + cols) + 2 * c;
            const float4 g0 = __ldcs(pg), g1 = __ldcs(pg + 1), u0 = __ldcs(pu), u1 = __ldcs(pu + 1);
            const uint4 dq = __ldcs(reinterpret_cast<const uint4 *>(dout + m * ldd) + c);
            const float g[8] = {g0.x, g0.y, g0.z, g0.w, g1.x, g1.y, g1.z, g1.w};
            const float u[8] = {u0.x, u0.y, u0.z, u0.w, u1.x, u1.y, u1.z, u1.w};
            const uint32_t dw[4] = {dq.x, dq.y, dq.z, dq.w};
            uint32_t wg[4], wu[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                float a0, b0, a1, b1;
                glu_gradients(g[2 * j], u[2 * j], bf16_lo(dw[j]), a0, b0);
                glu_gradients(g[2 * j + 1], u[2 * j + 1], bf16_hi(dw[j]), a1, b1);
                wg[j] = pack_bf16x2(a0, a1);
                wu[j] = pack_bf16x2(b0, b1);
            }
            reinterpret_cast<uint4 *>(dg + m * ldo)[c] = make_uint4(wg[0], wg[1], wg[2], wg[3]);
            reinterpret_cast<uint4 *>(du + m * ldo)[c] = make_uint4(wu[0], wu[1], wu[2], wu[3]);
        } else {
            float a, b;
            glu_gradients(gu[m * ldgu + c], gu[m * ldgu + cols + c], bf16_to_f32(dout[m * ldd + c]), a, b);
            dg[m * ldo + c] = f32_to_bf16(a);
            du[m * ldo + c] = f32_to_bf16(b);
        }
    }
}

}  // namespace mbglu
